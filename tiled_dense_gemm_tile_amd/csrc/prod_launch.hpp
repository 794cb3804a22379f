// The choice of kernel for a product of prod.hpp, and its launch.
#pragma once

#include "prod_api.hpp"
#include "prod_mid.hpp"
#include "prod_rows.hpp"
#include "prod_w4.hpp"

namespace tg {

inline unsigned prod_tiles(ProdArgs &p, int bm, int bn) {
    p.tiles_m = (p.M + bm - 1) / bm;
    p.tiles_n = (p.N + bn - 1) / bn;
    p.group_m = 4;
    return (unsigned)(p.tiles_m * (int64_t)p.tiles_n);
}

inline int64_t tiles_of(const ProdArgs &p, int bm, int bn) {
    return ((p.M + bm - 1) / bm) * (int64_t)((p.N + bn - 1) / bn);
}

template <int T, int BM, int BN, int S, int KS, bool PAIR, bool ANY, class Epi>
hipError_t go_mid(ProdArgs p, const Epi &e, hipStream_t s) {
    const unsigned grid = prod_tiles(p, BM, PAIR ? BN / 2 : BN);
    hipLaunchKernelGGL((prod_mid_kernel<T, BM, BN, ANY ? 2 : S, KS, PAIR, ANY, Epi>), dim3(grid), dim3(256 * KS), 0, s, p,
                       e);
    return hipGetLastError();
}

// 256 x 256 tiles in whole rounds of one a CU; what is left of up to half a
// round in 128 x 128 tiles (four times as many: weight gradients of 8192 x 8256
// x 4096, 16 tiles past four rounds, 973 -> 917 us).  8-bit operands without the
// lines brought ahead (8192 x 14336 x 4096 359 us, with them 364: more than two
// runs in turn differ, less than two cards; the gradients' products gain, 3280 ->
// 3020, the gated block neither way, 1356 without, 1348 with).
template <int T, bool PAIR, class Epi>
hipError_t go_w4(ProdArgs p, const Epi &e, hipStream_t s) {
    const unsigned tiles = prod_tiles(p, 256, PAIR ? 128 : 256), cus = 256, rest = tiles % cus;
    const bool cut = tiles > cus && rest > 0 && rest <= cus / 2;
    p.run = (int)(cut ? tiles - rest : tiles);
    hipLaunchKernelGGL((prod_w4_kernel<T, PAIR, T != kI8, Epi>), dim3(tiles < cus ? tiles : cus), dim3(256), 0, s, p, e);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !cut) return err;
    // (one a CU; more of them two a CU)
    if (rest <= cus / 4)
        hipLaunchKernelGGL((prod_mid_kernel<T, 128, 128, 2, 2, PAIR, false, Epi, true>), dim3(4 * rest), dim3(512), 0, s,
                           p, e);
    else
        hipLaunchKernelGGL((prod_mid_kernel<T, 128, 128, 2, 1, PAIR, false, Epi, true>), dim3(4 * rest), dim3(256), 0, s,
                           p, e);
    return hipGetLastError();
}

// 32 TM x 128 tiles (PAIR: 64 columns), one a CU.
template <int T, bool PAIR, int TM, class Epi>
hipError_t go_w4_once(ProdArgs p, const Epi &e, hipStream_t s) {
    p.run = (int)prod_tiles(p, 32 * TM, PAIR ? 64 : 128);
    hipLaunchKernelGGL((prod_w4_kernel<T, PAIR, true, Epi, 4, TM>), dim3(p.run), dim3(256), 0, s, p, e);
    return hipGetLastError();
}

// Tiles by how many of them there are (a K tile's loads bound a workgroup, 31
// to 44 bytes a clock and CU, until all CUs have work; times in us, int8 M x N x
// K or the gated block's M x F x K in bf16, of weights that no cache holds; F
// 14336: of one set, which the Infinity Cache keeps.  From HBM 64 rows take 51,
// 128 55, 256 73, 512 101).
template <int T, bool PAIR, bool ANY, class Epi>
hipError_t launch_prod_tiles(const ProdArgs &p, const Epi &e, hipStream_t s) {
    constexpr int D = PAIR ? 2 : 1;                    // a tile's columns of B for one of the results
    const int64_t t64 = tiles_of(p, 64, 64 / D), t128 = tiles_of(p, 128, 128 / D);
    if constexpr (!ANY) {
        // 256 x 256: more 128 x 128 tiles than run at once, two a CU (gated 512 x
        // 14336 x 4096, 224 tiles: 88 against 125; 256 x 14336 x 4096, 112 tiles:
        // 90 against 66)
        if (t128 > 512 && p.KB > 0) return go_w4<T, PAIR>(p, e, s);
    }
    // The smallest tiles of which every CU has one at most, K cut over the waves
    // (int8 40 x 4096 x 4096: 256 tiles of 32 x 32 7.8, of 32 x 64 9.4, of 64 x 64
    // 11.7; 77 x 4096 x 4096: 384 of 32 x 32 13.3, 192 of 32 x 64 9.6; gated 200 x
    // 2048 x 4096: 64 x 64 17.3, 32 x 64 27.0; int8 300 x 4096 x 4096: 64 x 128
    // 17.0, 64 x 64 21.5).  Through registers two groups are too many but for
    // the smallest and the widest (int8 40 x 4099 x 4100: 32 x 64 in one group
    // 11.6, two 12.5; 130 x 4099 x 4100: 64 x 64 13.8 either way).
    if constexpr (!PAIR)
        if (tiles_of(p, 32, 32) <= 256) return go_mid<T, 32, 32, 3, ANY ? 2 : 4, PAIR, ANY>(p, e, s);
    if (tiles_of(p, 32, 64 / D) <= 256) return go_mid<T, 32, 64, 4, ANY ? 1 : 2, PAIR, ANY>(p, e, s);
    // (rows for one 64-row tile only: larger ones would be part empty.  int8 48
    // x 65536 x 4096: 59.5, 128 x 128 72.7)
    if (p.M <= 64) return go_mid<T, 64, 64, 4, 1, PAIR, ANY>(p, e, s);
    if (t64 <= 256) return go_mid<T, 64, 64, 4, ANY ? 1 : 2, PAIR, ANY>(p, e, s);
    if (tiles_of(p, 64, 128 / D) <= 256) return go_mid<T, 64, 128, 3, 2, PAIR, ANY>(p, e, s);
    if constexpr (!ANY) {
        // 128 x 128, one a CU, in the large tiles' schedule (int8 1000 x 4096 x 4096
        // 20.8, K cut over two groups of waves 23.8; gated 128 x 14336 x 4096 39 and
        // 42, 1024 x 2048 x 256 6.8 and 6.6)
        if (t128 <= 256 && p.KB > 0) return go_w4_once<T, PAIR, 4>(p, e, s);
        // 256 x 128 on one round of CUs, for K that covers the longer way to the
        // first and the last K tile, and the results' stores by half the waves
        // (K tiles of 128 bytes; int8 2000 x 4096 x 4096 33.8 us, 128 x 128 43.7;
        // gated 256 x 14336 x 4096 58 and 73, 2048 x 2048 x 2048 32 and 38, x 512
        // 12.9 and 13.9, 1200 x 2048 x 256 9.3 and 8.8; results at any alignment:
        // int8 2000 x 4095 x 4096 36.8 and 44.0, with C x 1024 21.0 and 18.3)
        if (tiles_of(p, 256, 128 / D) <= 256 && p.KB > (e.vec ? 7 : 23) * 128) return go_w4_once<T, PAIR, 8>(p, e, s);
    }
    // two workgroups a CU (gated 1024 x 2736 x 1008: 19.2; four slots and one
    // workgroup 29.3, 64 x 64 28.4)
    return go_mid<T, 128, 128, 2, 1, PAIR, ANY>(p, e, s);
}

// Products whose operands lie aligned (the library's own copies).
template <int T, class Epi>
hipError_t launch_prod_aligned(const ProdArgs &p, const Epi &e, hipStream_t s) {
    return launch_prod_tiles<T, false, false, Epi>(p, e, s);
}

// About how long such a product takes by itself, in us: enough to tell which of
// launch_prod_two's forms ends sooner (81 sizes of 600 to 8192: the one taken was
// never 3 % behind the other).
inline double prod_estimate(const ProdArgs &p) {
    const double k = (p.KB + 127) / 128;
    if (tiles_of(p, 64, 64) <= 256) return 0.4 * k;
    const int64_t t128 = tiles_of(p, 128, 128), t256 = tiles_of(p, 256, 256), rest = t256 % 256;
    if (t128 <= 512) return (t128 <= 256 ? 0.75 : 1.1) * k;
    return 1.41 * k * ((double)(t256 / 256) + (rest == 0 ? 0 : t256 < 256 || rest > 128 ? 1 : rest > 64 ? 0.75 : 0.5));
}

// Two such products (D NULL: left out).  One launch of 256 x 256 tiles, each
// product on a share of the CUs, takes longer for a K tile (1.57 us in place of
// 1.41: two sets of panels share the L2s), but leaves no CU idle in a last round
// and suits a product with too few tiles for the GPU (gradients of 4096 x 6000 x
// 2048: 403 us, one after the other 478; 8192 x 1000 x 4096 267 and 296; 3000 x
// 2000 x 1504 103 and 121; 8192 x 14336 x 4096, whose tiles fill whole rounds,
// 3281 and 3043).
template <int T, class Epi0, class Epi1>
hipError_t launch_prod_two(const ProdArgs &p0, const Epi0 &e0, const ProdArgs &p1, const Epi1 &e1, hipStream_t s) {
    ProdPair q;
    q.p[0] = p0;
    q.p[1] = p1;
    q.split = 128;
    const int64_t k0 = (p0.KB + 127) / 128, k1 = (p1.KB + 127) / 128;
    const int64_t few = tiles_of(p0, 64, 64) + tiles_of(p1, 64, 64);
    // Small ones in 64 x 64 tiles: a launch less (gradients of 64 x 64 x 64 10.5
    // us, 13.5 in two; 179 x 768 x 1768, 756 tiles of 24 and 3 K tiles, 18.0 and
    // 22.8; 2 x 1792 x 189, 56 K tiles, 17.5 and 16.0).
    if (few <= 1024 && k0 <= 32 && k1 <= 32) {
        const unsigned n0 = prod_tiles(q.p[0], 64, 64), n1 = prod_tiles(q.p[1], 64, 64);
        q.split = e0.D[0] ? (int)n0 : 0;
        const dim3 grid(q.split + (e1.D[0] ? n1 : 0));
        if (few <= 256)
            hipLaunchKernelGGL((prod_mid_two_kernel<T, 64, 64, 4, 2, Epi0, Epi1>), grid, dim3(512), 0, s, q, e0, e1);
        else
            hipLaunchKernelGGL((prod_mid_two_kernel<T, 64, 64, 4, 1, Epi0, Epi1>), grid, dim3(256), 0, s, q, e0, e1);
        return hipGetLastError();
    }
    if (!e0.D[0] || !e1.D[0])
        return e0.D[0] ? launch_prod_aligned<T>(p0, e0, s) : launch_prod_aligned<T>(p1, e1, s);
    const int64_t a = prod_tiles(q.p[0], 256, 256), b = prod_tiles(q.p[1], 256, 256);
    int64_t best = INT64_MAX;                          // the share that lets the later one end soonest
    for (int n = 8; n < 256; n += 8) {
        const int64_t x = (a + n - 1) / n * k0, y = (b + 255 - n) / (256 - n) * k1, end = x > y ? x : y;
        if (end < best) best = end, q.split = n;
    }
    if (k0 > 0 && k1 > 0 && 1.57 * (double)best < prod_estimate(p0) + prod_estimate(p1)) {
        q.p[0].run = (int)a;
        q.p[1].run = (int)b;
        hipLaunchKernelGGL((prod_w4_two_kernel<T, Epi0, Epi1>), dim3(256), dim3(256), 0, s, q, e0, e1);
        return hipGetLastError();
    }
    const hipError_t err = launch_prod_aligned<T>(p0, e0, s);
    return err != hipSuccess ? err : launch_prod_aligned<T>(p1, e1, s);
}

template <int T, int MB, bool PAIR, class Epi>
hipError_t go_rows(const ProdArgs &p, const Epi &e, hipStream_t s) {
    hipLaunchKernelGGL((prod_rows_kernel<T, MB, PAIR, Epi>), dim3((unsigned)((p.N + 15) / 16)), dim3(512), 0, s, p, e);
    return hipGetLastError();
}

// Any operands.
template <int T, bool PAIR, class Epi>
hipError_t launch_prod(const ProdArgs &p, const Epi &e, hipStream_t s) {
    // A few rows (every workgroup of prod_rows reads all of A, which from nine
    // rows on costs more than a tile's detour through LDS where the tiles fill
    // the GPU: int8 1 x 65536 x 4096 49 us against 57, 16 rows 63 against 58, 1 x
    // 4096 x 4096 5.4 against 7.5, 32 x 14336 x 4096 24 against 16; gated 1 x
    // 4096 x 4096 15.0 against 17.8, 32 rows 21.0 against 22.3)
    const int64_t t64 = tiles_of(p, 64, PAIR ? 32 : 64);
    if (p.M <= 8 || (p.M <= 16 && t64 < 200)) return go_rows<T, 1, PAIR>(p, e, s);
    if (p.M <= 32 && t64 <= 128) return go_rows<T, 2, PAIR>(p, e, s);
    if (tg_api::prod_aligned(p)) return launch_prod_tiles<T, PAIR, false, Epi>(p, e, s);
    return launch_prod_tiles<T, PAIR, true, Epi>(p, e, s);
}

}  // namespace tg
