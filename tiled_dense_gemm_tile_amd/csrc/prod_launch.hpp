// The choice of kernel for a product of prod.hpp, and its launch.
#pragma once

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

// Direct loads: rows on 16 bytes and whole 16-byte chunks.
inline bool prod_aligned(const ProdArgs &p) {
    auto on16 = [](const void *q, int64_t ld, int rows) {
        return (uintptr_t)q % 16 == 0 && (ld % 16 == 0 || rows == 1);
    };
    return p.KB % 16 == 0 && on16(p.A, p.lda, p.M) && on16(p.B, p.ldb, p.N) && (!p.B1 || on16(p.B1, p.ldb1, p.N));
}

// 256 x 256 tiles: from half a wave of them on.
template <int T, bool PAIR, class Epi>
bool launch_prod_w4(ProdArgs p, const Epi &e, hipStream_t s) {
    const unsigned tiles = prod_tiles(p, 256, PAIR ? 128 : 256), cus = 256;
    if (tiles < cus / 2 || p.KB == 0) return false;
    hipLaunchKernelGGL((prod_w4_kernel<T, PAIR, Epi>), dim3(tiles < cus ? tiles : cus), dim3(256), 0, s, p, e);
    return true;
}

template <int T, bool PAIR, bool ANY, class Epi>
hipError_t launch_prod_mid(ProdArgs p, const Epi &e, hipStream_t s) {
    if constexpr (!ANY)
        if (launch_prod_w4<T, PAIR>(p, e, s)) return hipGetLastError();
    const int64_t t128 = ((p.M + 127) / 128) * (int64_t)((p.N + (PAIR ? 63 : 127)) / (PAIR ? 64 : 128));
    if (t128 >= 200) {
        const unsigned grid = prod_tiles(p, 128, PAIR ? 64 : 128);
        hipLaunchKernelGGL((prod_mid_kernel<T, 128, 128, ANY ? 2 : 4, PAIR, ANY, Epi>), dim3(grid), dim3(256), 0, s, p, e);
    } else {
        const unsigned grid = prod_tiles(p, 64, PAIR ? 32 : 64);
        hipLaunchKernelGGL((prod_mid_kernel<T, 64, 64, ANY ? 2 : 4, PAIR, ANY, Epi>), dim3(grid), dim3(256), 0, s, p, e);
    }
    return hipGetLastError();
}

// Products whose operands lie aligned (the library's own copies).
template <int T, class Epi>
hipError_t launch_prod_aligned(const ProdArgs &p, const Epi &e, hipStream_t s) {
    return launch_prod_mid<T, false, false, Epi>(p, e, s);
}

// Any operands.
template <int T, bool PAIR, class Epi>
hipError_t launch_prod(ProdArgs p, const Epi &e, hipStream_t s) {
    if (p.M <= 32) {
        const unsigned grid = (unsigned)((p.N + 15) / 16);
        if (p.M <= 16)
            hipLaunchKernelGGL((prod_rows_kernel<T, 1, PAIR, Epi>), dim3(grid), dim3(512), 0, s, p, e);
        else
            hipLaunchKernelGGL((prod_rows_kernel<T, 2, PAIR, Epi>), dim3(grid), dim3(512), 0, s, p, e);
        return hipGetLastError();
    }
    if (prod_aligned(p)) return launch_prod_mid<T, PAIR, false, Epi>(p, e, s);
    return launch_prod_mid<T, PAIR, true, Epi>(p, e, s);
}

}  // namespace tg
