// Weight gradient from block-scaled rows: D = A^T.B + C, A (K x M) bf16, B
// (K x N) e4m3 codes with one e8m0 scale per 32 columns of a row.
//
// The kernel that takes every call: 128 x 128 output tiles, K tiles of 32
// rows, four waves of 64 x 64.  Both operands lie MN-contiguous, so their K
// tiles are staged in LDS as they lie (rows of 128 elements) and MFMA
// fragments -- eight K-consecutive values of one column -- come from gfx950's
// transposing LDS read.  B's codes become bf16 on the way into LDS, where 16
// consecutive columns of a row share one scale (a fragment's eight values
// have eight scales); e4m3 * 2^e is exact in bf16.  Rows may start at any
// element: loads are 16-byte vectors of element alignment.  Bound by the wait
// for each K tile's loads, one tile ahead (4090 x 4096 x 4100 315 us, 436
// TFLOP/s): large calls whose rows start off 16 bytes copy A and run the
// four-wave kernel.
#pragma once

#include "common.hpp"
#include "gemm_f16.hpp"
#include "rows.hpp"

namespace tg {

struct WgradArgs {
    const void *A, *B;
    const uint8_t *SF;
    const void *C;
    void *D;
    int64_t lda, ldb, ldsf, ldc, ldd;
    int M, N, K;
    int tiles_m, tiles_n, group_m;
    // K cut into ranges of k_split rows: range s writes its fp32 partial tile
    // to the M x ldw matrix at ws + s * M * ldw (ws null: uncut)
    int k_split;
    float *ws;
    int64_t ldw;
};

// 16 e4m3 codes with their scale as bf16.
__device__ __forceinline__ void fp8_up(u32x4 q, uint32_t code, u32x4 &lo, u32x4 &hi) {
    const float scale = __builtin_bit_cast(float, code << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], scale, false));
        const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], scale, true));
        if (i < 2) {
            lo[2 * i] = a;
            lo[2 * i + 1] = b;
        } else {
            hi[2 * i - 4] = a;
            hi[2 * i - 3] = b;
        }
    }
}

// Four columns of D = v + C, at any element alignment.
template <bool OUT_BF16>
__device__ __forceinline__ void wgrad_put(f32x4 v, const void *C, int64_t ldc, void *D, int64_t ldd, int m, int n) {
    struct __attribute__((packed, aligned(4))) F4 {
        f32x4 v;
    };
    struct __attribute__((packed, aligned(2))) H4 {
        u32x2 v;
    };
    if constexpr (OUT_BF16) {
        if (C) {
            const u32x2 c = ((const H4 *)((const uint16_t *)C + (int64_t)m * ldc + n))->v;
            v[0] += __builtin_bit_cast(float, c[0] << 16);
            v[1] += __builtin_bit_cast(float, c[0] & 0xffff0000u);
            v[2] += __builtin_bit_cast(float, c[1] << 16);
            v[3] += __builtin_bit_cast(float, c[1] & 0xffff0000u);
        }
        ((H4 *)((uint16_t *)D + (int64_t)m * ldd + n))->v = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
        if (C) v += ((const F4 *)((const float *)C + (int64_t)m * ldc + n))->v;
        ((F4 *)((float *)D + (int64_t)m * ldd + n))->v = v;
    }
}

// A with its rows moved to 16-byte boundaries, for the four-wave kernel: a
// workgroup copies 2048 columns of a row.
__global__ void __launch_bounds__(256)
    wgrad_align_kernel(const void *A, int64_t lda, void *out, int64_t ldo, int K, int M) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= M) return;
    for (int64_t k = blockIdx.y; k < K; k += gridDim.y)   // (out: whole vectors, ldo >= c + 8)
        *(RowVec<1>::V *)((__bf16 *)out + k * ldo + c) = RowVec<1>::load((const __bf16 *)A + k * lda, c, M);
}

typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

template <bool OUT_BF16>
__global__ void __launch_bounds__(256) gemm_wgrad_any_kernel(WgradArgs p) {
    constexpr int BM = 128, BN = 128, KT = 32;
    constexpr int PITCH = 272;                         // LDS row: 128 bf16, and 16 bytes that spread rows over banks
    constexpr int OPERAND = KT * PITCH, SLOT = 2 * OPERAND;
    __shared__ __attribute__((aligned(16))) char smem[2 * SLOT];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    int tmi, tni, split = 0;
    if (p.ws)
        tile_order_split(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, tmi, tni, split);
    else
        tile_order(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    const int m0 = tmi * BM, n0 = tni * BN;
    const int64_t k_lo = (int64_t)split * p.k_split;
    const int64_t k_hi = p.ws ? (k_lo + p.k_split < p.K ? k_lo + p.k_split : p.K) : p.K;

    // A: thread t loads rows t / 16 and t / 16 + 16, columns 8 (t % 16) .. + 7;
    // B: row t / 8, columns 16 (t % 8) .. + 15
    const int ar = tid >> 4, ac = m0 + (tid & 15) * 8;
    const int br = tid >> 3, bc = n0 + (tid & 7) * 16;
    u32x4 va[2], vb;
    uint32_t code;
    struct __attribute__((packed, aligned(1))) Q16 {
        u32x4 v;
    };
    auto load = [&](int64_t k) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = k + ar + 16 * h;
            va[h] = u32x4{0u, 0u, 0u, 0u};
            if (row < k_hi && ac < p.M)
                va[h] = __builtin_bit_cast(u32x4, RowVec<1>::load((const __bf16 *)p.A + row * p.lda, ac, p.M));
        }
        const int64_t row = k + br;
        vb = u32x4{0u, 0u, 0u, 0u};
        code = 127u;
        if (row < k_hi && bc < p.N) {                  // N % 32 == 0: whole vectors
            vb = ((const Q16 *)((const uint8_t *)p.B + row * p.ldb + bc))->v;
            code = p.SF[row * p.ldsf + bc / 32];
        }
    };
    auto store = [&](int slot) __attribute__((always_inline)) {
        char *sA = smem + slot * SLOT, *sB = sA + OPERAND;
#pragma unroll
        for (int h = 0; h < 2; ++h) *(u32x4 *)(sA + (ar + 16 * h) * PITCH + (tid & 15) * 16) = va[h];
        u32x4 lo, hi;
        fp8_up(vb, code, lo, hi);
        *(u32x4 *)(sB + br * PITCH + (tid & 7) * 32) = lo;
        *(u32x4 *)(sB + br * PITCH + (tid & 7) * 32 + 16) = hi;
    };

    // Transposing reads: lane (group g = l / 16, i = l % 16) reads row 8 g + 4 h
    // + i / 4, columns 4 (i % 4) .. + 3 of a block of 16 and receives column
    // i's rows 8 g + 4 h .. + 3.
    const int fr = lane & 15, fq = lane >> 4;
    const int frag = (8 * fq + (fr >> 2)) * PITCH + (fr & 3) * 8;
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    auto read = [&](const char *s, int block) __attribute__((always_inline)) {
        const char *a = s + frag + block * 32;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)a);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(a + 4 * PITCH));
        const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
        return u32x4{l2[0], l2[1], h2[0], h2[1]};
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (k_lo < k_hi) {
        load(k_lo);
        store(0);
    }
    __syncthreads();
    int slot = 0;
    for (int64_t k = k_lo; k < k_hi; k += KT, slot ^= 1) {
        const bool more = k + KT < k_hi;
        if (more) load(k + KT);
        const char *sA = smem + slot * SLOT, *sB = sA + OPERAND;
        u32x4 fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[i] = read(sA, wm * 4 + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[j] = read(sB, wn * 4 + j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32<false>(fb[j], fa[i], acc[i][j]);
        if (more) store(slot ^ 1);
        __syncthreads();
    }

    // Block (i, j) holds its transpose: lane l has row 16 i + l % 16 of the
    // wave's 64 and columns 16 j + 4 (l / 16) .. + 3 (whole vectors, N % 32 == 0).
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + wm * 64 + 16 * i + fr;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + wn * 64 + 16 * j + 4 * fq;
            if (n >= p.N) continue;
            const f32x4 v = acc[i][j];
            if (p.ws) {
                *(f32x4 *)(p.ws + ((int64_t)split * p.M + m) * p.ldw + n) = v;
            } else {
                wgrad_put<OUT_BF16>(v, p.C, p.ldc, p.D, p.ldd, m, n);
            }
        }
    }
}

}  // namespace tg
