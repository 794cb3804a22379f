// Products of a few rows (up to 32) with a large matrix: bound by the reading
// of that matrix (gated 1 x 14336 x 4096 42.3 us, 5.5 TB/s; int8 1 x 4096 x 14336
// 10.6), so nothing of it passes through LDS.  (32 columns a workgroup,
// units of 64 and 128 bytes, and streaming loads were slower: int8 1 x 4096 x
// 14336 13.0 us; 16.3, 12.8 to 16.3 and 14.7.)
//
// A workgroup of eight waves owns 16 result columns (PAIR: 16 gate and 16 up
// rows of the weights) and cuts K over its waves in units of 256 bytes: wave w
// takes units w, w + 8, ...  Lane l loads 16 bytes of weight row l % 16 at byte
// 64 s + 16 (l / 16) of the unit, s = 0 .. 3, and the same bytes of row l % 16
// of A, and multiplies them as they came: no exchange, no wait but for the
// loads.  A wave loads a unit ahead.  The waves' sums meet in LDS and are
// added in order.
#pragma once

#include "prod.hpp"

namespace tg {

// MB: blocks of 16 rows of A.
template <int T, int MB, bool PAIR, class Epi>
__global__ void __launch_bounds__(512) prod_rows_kernel(ProdArgs p, Epi e) {
    constexpr int RB = PAIR ? 2 : 1, NW = 8, UNIT = 256;
    __shared__ __attribute__((aligned(16))) float red[NW][MB * RB][256];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    // (rows past the end are read as the last one: their results are not stored)
    const int n = n0 + r < p.N ? n0 + r : p.N - 1;
    const char *w[RB];
    w[0] = (const char *)p.B + (int64_t)n * p.ldb;
    if constexpr (PAIR) w[1] = (const char *)p.B1 + (int64_t)n * p.ldb1;
    const char *x[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int m = 16 * b + r < p.M ? 16 * b + r : p.M - 1;
        x[b] = (const char *)p.A + (int64_t)m * p.lda;
    }
    f32x4 acc[MB][RB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int c = 0; c < RB; ++c) acc[b][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    u32x4 wf[2][RB][4], xf[2][MB][4];
    auto load = [&](int buf, int unit) __attribute__((always_inline)) {
        const int kb = unit * UNIT + 16 * q;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int c = 0; c < RB; ++c) wf[buf][c][s] = load_chunk_whole<T>(w[c] + kb + 64 * s);
#pragma unroll
            for (int b = 0; b < MB; ++b) xf[buf][b][s] = load_chunk_whole<T>(x[b] + kb + 64 * s);
        }
    };
    auto multiply = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int c = 0; c < RB; ++c) acc[b][c] = prod_mfma<T>(wf[buf][c][s], xf[buf][b][s], acc[b][c]);
    };
    const int whole = p.KB / UNIT;
    int u = wave;
    if (u < whole) load(0, u);
    while (u < whole) {
        if (u + NW < whole) load(1, u + NW);
        multiply(0);
        u += NW;
        if (u >= whole) break;
        if (u + NW < whole) load(0, u + NW);
        multiply(1);
        u += NW;
    }
    // the last unit, if K ends inside it: one wave's, 64 bytes at a time
    if (p.KB % UNIT != 0 && u == whole) {
        for (int kb = whole * UNIT; kb < p.KB; kb += 64) {
            const int at = kb + 16 * q;
            u32x4 xl[MB], wl[RB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                xl[b] = u32x4{0u, 0u, 0u, 0u};
                if (at < p.KB) xl[b] = load_chunk<T>(x[b], at, p.KB);
            }
#pragma unroll
            for (int c = 0; c < RB; ++c) {
                wl[c] = u32x4{0u, 0u, 0u, 0u};
                if (at < p.KB) wl[c] = load_chunk<T>(w[c], at, p.KB);
            }
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int c = 0; c < RB; ++c) acc[b][c] = prod_mfma<T>(wl[c], xl[b], acc[b][c]);
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int c = 0; c < RB; ++c) *(f32x4 *)&red[wave][b * RB + c][lane * 4] = acc[b][c];
    __syncthreads();
    // result (m, n0 + i): lane 16 (i / 4) + m % 16, register i % 4
    if (threadIdx.x >= MB * 256) return;
    const int b = threadIdx.x >> 8, m = 16 * b + ((threadIdx.x >> 4) & 15), i = threadIdx.x & 15;
    const int at = (16 * (i >> 2) + (m & 15)) * 4 + (i & 3);
    if (m >= p.M || n0 + i >= p.N) return;
    if constexpr (T == kI8) {
        int32_t s = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) s += __builtin_bit_cast(int32_t, red[k][b][at]);
        e.one(m, n0 + i, s);
    } else {
        float s[RB];
#pragma unroll
        for (int c = 0; c < RB; ++c) {
            s[c] = red[0][b * RB + c][at];
#pragma unroll
            for (int k = 1; k < NW; ++k) s[c] += red[k][b * RB + c][at];
        }
        e.one(m, n0 + i, s[0], s[RB - 1]);
    }
}

}  // namespace tg
