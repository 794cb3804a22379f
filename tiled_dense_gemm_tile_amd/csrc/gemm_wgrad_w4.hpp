// Weight gradient from block-scaled rows, four-wave kernel: 256 x 256 output
// tiles, K tiles of 64 rows, for 16-byte rows of A and B.
//
// The MFMA schedule is the 16-bit four-wave kernel's (gemm_f16_w4.hpp: waves
// of 128 x 128 in 8 x 8 accumulator blocks, K steps of 32, the second step of
// a K tile multiplied after the next tile's barrier) with both operands
// MN-contiguous: a K tile lies in LDS as 64 rows of 256 bf16 and fragments are
// read with ds_read_b64_tr_b16.  A's tile comes by direct global -> LDS loads.
// B's tile is half as many bytes in memory and takes the registers: each
// thread loads 64 codes of a row and its scales a K tile ahead, converts them
// (one instruction per two, with the scale) between the MFMAs of a tile's
// second half, and writes them into the slot that the tile before has left.
// A fragment's eight K-consecutive values have eight different scales, which
// is why the conversion comes before LDS and not after it.
//
// Tiles past the last full round of 256 workgroups (all of them, in a small
// grid) may be cut along K into `splits` ranges, whose fp32 partial tiles go
// to the workspace for a second kernel to add in order.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "gemm_f16_w4.hpp"
#include "gemm_wgrad.hpp"
#include "pipeline.hpp"

namespace tg {

struct Wgrad4Args {
    const void *A, *B;
    const uint8_t *SF;
    const void *C;
    void *D;
    int64_t lda, ldb, ldsf, ldc, ldd;
    int M, N, K;
    int tiles_m, tiles_n, group_m;
    int full;                                          // tiles multiplied whole: the first `full` of the walk
    int splits, k_split;                               // of the others: ranges, and K per range
    float *ws;                                         // range s of tile full + i at ws + (s * rest + i) * 65536
};

// Tile `id` of the walk in groups of group_m tile rows.
__device__ __forceinline__ void walk_tile(int id, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
    const int group_size = group_m * tiles_n;
    const int group = id / group_size;
    const int first_m = group * group_m;
    const int gm = (tiles_m - first_m) < group_m ? (tiles_m - first_m) : group_m;
    const int in_group = id - group * group_size;
    tm = first_m + in_group % gm;
    tn = in_group / gm;
}

// Renumbering that gives each of the eight XCDs a run of ids.
__device__ __forceinline__ int xcd_order(int wg, int nwg) {
    const int q = nwg >> 3, r = nwg & 7, x = wg & 7;
    return x * q + (x < r ? x : r) + (wg >> 3);
}

// LDS operations outstanding when block row i of a tile's second half needs
// its first-half fragments (gemm_f16_w4.hpp, tr_row_wait), with the writes of
// converted B that the half has issued before its MFMA 8 i (two after each
// 16 MFMAs' fourth conversion: see kConvert below).
constexpr int wgrad_writes_before(int q) {
    int n = 0;
    for (int s = 0; s < 16; ++s)
        if (s % 2 == 1 && 4 * s + 2 < q) ++n;
    return n;
}
constexpr int wgrad_row_wait(int i) {
    int n = (7 - i) * 2;
    const int issued = (8 * i + 2) / 3;
    for (int m = 0; m < issued && m < 16; ++m) n += 2;
    n += wgrad_writes_before(8 * i);
    return n > 15 ? 15 : n;
}

template <bool OUT_BF16>
__global__ void __launch_bounds__(256) gemm_wgrad_w4_kernel(Wgrad4Args p, F16Epi e) {
    constexpr int TM = 8, TN = 8, BM = 256, BN = 256, KT = 64;
    constexpr int WTM = 128, WTN = 128, Q = TM * TN;
    constexpr int SLOT = KT * 512;                     // 64 rows of 256 bf16
    constexpr int B_BASE = 2 * SLOT;
    constexpr int RING_BYTES = 4 * SLOT;
    constexpr int EPI_BYTES = 4 * 32 * (WTN + 8) * 4;
    static_assert(EPI_BYTES <= RING_BYTES && RING_BYTES <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[RING_BYTES];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int rest = p.tiles_m * p.tiles_n - p.full;
    int tmi, tni, split = -1, part = 0;
    if ((int)blockIdx.x < p.full) {
        walk_tile(xcd_order(blockIdx.x, p.full), p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    } else {
        const int id = xcd_order(blockIdx.x - p.full, rest * p.splits);
        split = id / rest;
        part = id - split * rest;
        walk_tile(p.full + part, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    }
    const int m0 = tmi * BM, n0 = tni * BN;
    const int M = p.M, N = p.N;
    const int k_lo = split > 0 ? split * p.k_split : 0;
    const int K = split < 0 ? p.K : (p.K - k_lo < p.k_split ? p.K - k_lo : p.k_split);
    const int nt = (K + KT - 1) / KT;

    // ---- A: direct global -> LDS, as gemm_f16_w4t_kernel's AT operand
    const char *a_base = (const char *)p.A + (int64_t)k_lo * p.lda * 2;
    uint32_t a_off[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = 2 * (4 * j + wave) + (lane >> 5);
        const int lchk = ((lane & 31) >> 1) ^ (row & 3) ^ (((row >> 3) & 1) << 2);
        a_off[j] = (uint32_t)((row * p.lda + lchk * 16 + (lane & 1) * 8) * 2);
    }
    auto dma_a = [&](int t, int j) __attribute__((always_inline)) {
        const int k0 = t * KT;
        const uint32_t span = (span_bytes(K - k0, M - m0, p.lda, 2) + 15u) & ~15u;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(a_base + ((int64_t)k0 * p.lda + m0) * 2, span);
        dma_load<16>(r, smem + (t & 1) * SLOT + (j * 4 + wave) * 1024, a_off[j]);
    };

    // ---- B: thread t holds row t / 4 of a K tile, columns 16 (t % 4) + 64 j
    // .. + 15, and the eight scales of the row's 256 columns (of its last
    // eight blocks where N ends inside the tile: s_shift bits too far left;
    // rows past K take the last row's, with codes 0)
    const int br = tid >> 2, bt = tid & 3;
    const uint32_t b_off = (uint32_t)(br * p.ldb) + bt * 16;
    const int nb = N / 32, s_at = n0 / 32 < nb - 8 ? n0 / 32 : nb - 8, s_shift = 8 * (n0 / 32 - s_at);
    const char *b_base = (const char *)p.B + (int64_t)k_lo * p.ldb + n0;
    const uint8_t *s_base = p.SF + (int64_t)k_lo * p.ldsf + s_at;
    struct __attribute__((packed, aligned(1))) U64 {
        uint64_t v;
    };
    u32x4 vb[4];
    uint64_t vs;
    auto load_b = [&](int t, int j) __attribute__((always_inline)) {
        const int k0 = t * KT;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(b_base + (int64_t)k0 * p.ldb, span_bytes(K - k0, N - n0, p.ldb, 1));
        vb[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, b_off + 64 * j, 0, 0));
    };
    auto load_s = [&](int t) __attribute__((always_inline)) {
        const int row = t * KT + br < K ? t * KT + br : K - 1;
        vs = ((const U64 *)(s_base + (int64_t)row * p.ldsf))->v;
    };
    // Vector j converted, four columns a step; written as two 16-byte halves.
    // (LDS row br, 32-byte chunk bt + 4 j at ^ (br % 4) ^ 4 (br / 8 % 2), the
    // layout of A's slots)
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    uint32_t b_put[2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
        b_put[o] = lds0 + B_BASE + br * 512 + ((bt ^ (br & 3)) + 4 * (o ^ ((br >> 3) & 1))) * 32;
    uint32_t sc[2];                                    // scales of this thread's vectors 0, 1 and 2, 3, in bytes 0 and 2
    auto take_scales = [&]() __attribute__((always_inline)) {
        const uint64_t s = (vs >> s_shift) >> (8 * (bt >> 1));
        sc[0] = (uint32_t)s;
        sc[1] = (uint32_t)(s >> 32);
    };
    u32x4 half;
    auto convert = [&](auto step, int slot) __attribute__((always_inline)) {
        constexpr int j = decltype(step)::value / 4, i = decltype(step)::value % 4;
        const float scale = __builtin_bit_cast(
            float, (j & 1) ? (sc[j / 2] & 0xff0000u) << 7 : (sc[j / 2] & 0xffu) << 23);
        half[2 * (i & 1)] =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vb[j][i], scale, false));
        half[2 * (i & 1) + 1] =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vb[j][i], scale, true));
        if constexpr (i & 1) {
            const uint32_t at = b_put[j & 1] + slot * SLOT;
            if constexpr (i == 1)
                asm volatile("ds_write_b128 %0, %1 offset:%c2" : : "v"(at), "v"(half), "n"(256 * (j / 2)) : "memory");
            else
                asm volatile("ds_write_b128 %0, %1 offset:%c2" : : "v"(at), "v"(half), "n"(256 * (j / 2) + 16) : "memory");
        }
    };

    // ---- fragments: transposing reads (gemm_f16_w4t_kernel, MN-contiguous)
    const int fr = lane & 15, fq = lane >> 4;
    auto mn_base = [&](int wb, int b) __attribute__((always_inline)) {
        const int g = (fr >> 2) ^ ((fq & 1) << 2);
        return lds0 + (8 * fq + (fr >> 2)) * 512 + (wb * 8 + (b ^ g)) * 32 + (fr & 3) * 8;
    };
    uint32_t a_mn[TM], b_mn[TN];
#pragma unroll
    for (int b = 0; b < TM; ++b) a_mn[b] = mn_base(wm, b);
#pragma unroll
    for (int b = 0; b < TN; ++b) b_mn[b] = B_BASE + mn_base(wn, b);
    auto ldfrag_tr = [&](uint32_t a) __attribute__((always_inline)) {
        u32x2 lo, hi;
        asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(lo) : "v"(a));
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:2048" : "=v"(hi) : "v"(a));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    f32x4 acc[TM][TN];
    u32x4 fa[2][TM], fb[2][TN];                        // [K step][block]
    auto read_frag = [&](int t, int st, int k) __attribute__((always_inline)) {
        const uint32_t o = (t & 1) * SLOT + st * 32 * 512;
        if (k == 0 || k > TN) {
            const int i = k == 0 ? 0 : k - TN;
            fa[st][i] = ldfrag_tr(a_mn[i] + o);
        } else {
            fb[st][k - 1] = ldfrag_tr(b_mn[k - 1] + o);
        }
    };
    auto mfma = [&](auto zero, int st, int i, int j) __attribute__((always_inline)) {
        if constexpr (decltype(zero)::value)
            mfma16_zero_asm<false>(acc[i][j], fb[st][j], fa[st][i]);
        else
            mfma16_acc_asm<false>(acc[i][j], fb[st][j], fa[st][i]);
        __builtin_amdgcn_sched_barrier(0);
    };

    // One K tile.  First half: step 1 of tile t - 1, with the reads of tile t
    // step 0 and the loads of A(t + 1).  Second half: step 0 of tile t, with
    // the reads of step 1, the conversion of B(t + 1) (a step of two
    // instructions per four MFMAs, a write per eight) and, as its registers
    // fall free, the loads of B(t + 2), which have until the next tile's
    // second half to land.
    auto tile = [&](auto first, int t) __attribute__((always_inline)) {
        constexpr int RD = TM + TN;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (!decltype(first)::value) mfma(std::false_type(), 1, q / TN, q % TN);
            if (q * RD % Q == 0 && q * RD / Q < RD) read_frag(t, 0, q * RD / Q);
            if (q % 8 == 2) dma_a(t + 1, q / 8);
        }
        static_for<0, Q>([&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q % TN == 0) __builtin_amdgcn_s_waitcnt(0xC07F | (wgrad_row_wait(q / TN) << 8));
            mfma(first, 0, q / TN, q % TN);
            if constexpr (q % 3 == 0 && q / 3 < TM + TN) read_frag(t, 1, q / 3);
            if constexpr (q == 1) take_scales();
            if constexpr (q % 4 == 2) {
                convert(std::integral_constant<int, q / 4>(), (t + 1) & 1);
                if constexpr (q / 4 % 4 == 3) load_b(t + 2, q / 16);
                if constexpr (q / 4 == 15) load_s(t + 2);
            }
        });
        wait_vmcnt<5>();                               // A(t + 1) landed; B(t + 2) and its scales may still run
        wait_lgkmcnt0();
        barrier();
    };

    if (nt > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dma_a(0, j);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_b(0, j);
        load_s(0);
        take_scales();
        static_for<0, 16>([&](auto s) __attribute__((always_inline)) { convert(s, 0); });
#pragma unroll
        for (int j = 0; j < 4; ++j) load_b(1, j);
        load_s(1);
        wait_vmcnt<5>();
        wait_lgkmcnt0();
        barrier();
        tile(std::true_type(), 0);
        for (int t = 1; t < nt; ++t) tile(std::false_type(), t);
#pragma unroll
        for (int q = 0; q < Q; ++q) mfma(std::false_type(), 1, q / TN, q % TN);
        mfma_result_fence<TM, TN>(acc);
    } else {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    barrier();
    if (split < 0) {
        epilogue_lds16t<OUT_BF16, TM, TN, WTM, WTN, kStoreStream>(acc, smem, wave, lane, wm, wn, m0, n0, M, N, p.C,
                                                                  p.ldc, p.D, p.ldd, e);
    } else {
        // a whole partial tile, 256 x 256 (stays cacheable: it is read next)
        float *out = p.ws + ((int64_t)split * rest + part) * 65536;
        F16Epi v;
        v.vec_c = false;
        v.vec_d = true;
        epilogue_lds16t<false, TM, TN, WTM, WTN, 0>(acc, smem, wave, lane, wm, wn, 0, 0, BM, BN, nullptr, 0, out, BN,
                                                    v);
    }
}

// D = the `splits` partial tiles of each cut tile added in order, plus C: four
// columns a thread, 64 threads a row, four rows a workgroup.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) wgrad_reduce_kernel(Wgrad4Args p) {
    const int rest = p.tiles_m * p.tiles_n - p.full;
    const int part = blockIdx.x >> 6, r = (blockIdx.x & 63) * 4 + (threadIdx.x >> 6), c = (threadIdx.x & 63) * 4;
    int tm, tn;
    walk_tile(p.full + part, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int m = tm * 256 + r, n = tn * 256 + c;
    if (m >= p.M || n >= p.N) return;                  // (N % 32 == 0: whole vectors)
    const float *w = p.ws + (int64_t)part * 65536 + r * 256 + c;
    const int64_t slice = (int64_t)rest * 65536;
    f32x4 s = *(const f32x4 *)w;
    int k = 1;
    for (; k + 4 <= p.splits; k += 4) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *(const f32x4 *)(w + (k + i) * slice);
#pragma unroll
        for (int i = 0; i < 4; ++i) s += v[i];
    }
    for (; k < p.splits; ++k) s += *(const f32x4 *)(w + k * slice);
    wgrad_put<OUT_BF16>(s, p.C, p.ldc, p.D, p.ldd, m, n);
}

}  // namespace tg
