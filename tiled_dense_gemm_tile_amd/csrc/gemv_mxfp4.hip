// C ABI and kernel of gemv_mxfp4 (include/tilegemm_ops.h): a few 16-bit rows
// times 4-bit weights with group scales.
//
// Bound by the reading of W (half a byte per weight; 2 M flops per weight).
// A workgroup takes 16 weight rows and its waves share K, so that a matrix
// of a few thousand rows still spreads over the whole GPU; each wave runs
// 16x16x32 MFMAs with X as the row operand (its M rows padded to 16) and the
// weights, converted to 16 bits with their scale by one instruction per two,
// as the column operand.  A lane's 16 bytes of a weight row are one whole
// 32-element block with one scale: K is permuted inside a step of 128 so
// that lane group g holds block g, and X is read with the same permutation.
// The waves' sums are joined through LDS in wave order.
#include "api.hpp"
#include "pipeline.hpp"
#include "rows.hpp"
#include "../../include/tilegemm_ops.h"

using namespace tg_api;

namespace tg {

struct GemvArgs {
    const void *X;
    const uint8_t *W, *SF;
    const void *C;
    void *D;
    int64_t ldx, ldw_bytes, ldsf, ldc, ldd;
    int M, N, K;
    int kshift;                                        // scale index of element k: k >> kshift
    int tiles_n;
};

constexpr int kGemvWaves = 8;

struct __attribute__((packed, aligned(1))) Bytes16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(2))) Halves8 {
    u32x4 v;
};

// 8 weights (one word of codes) with their scale as bf16 / fp16.
template <bool FP16>
__device__ __forceinline__ u32x4 fp4_up(uint32_t w, float scale) {
    u32x4 o;
    if constexpr (FP16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
    } else {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    }
    return o;
}

template <bool FP16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// fp16 x = hi + lo exactly, both bf16: hi holds its upper 8 significant bits,
// the remainder at most 3 (and bf16's exponents reach below fp16's).
__device__ __forceinline__ void split_f16(u32x4 x, u32x4 &hi, u32x4 &lo) {
    const f16x8 v = __builtin_bit_cast(f16x8, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = (float)v[2 * i], b = (float)v[2 * i + 1];
        hi[i] = pack_bf16x2(a, b);
        const float ra = a - __builtin_bit_cast(float, hi[i] << 16);
        const float rb = b - __builtin_bit_cast(float, hi[i] & 0xffff0000u);
        // (an infinity or NaN stays in hi alone)
        lo[i] = pack_bf16x2(__builtin_isfinite(a) ? ra : 0.0f, __builtin_isfinite(b) ? rb : 0.0f);
    }
}

// The waves' sums of block a (16 rows of X) joined in wave order, plus C, to D.
// red[wave][4 a + r][lane]: lane l, register r holds row 16 a + 4 (l / 16) + r
// and column l % 16.
template <bool OUT_BF16, int MB>
__device__ __forceinline__ void gemv_join(const float (&red)[kGemvWaves][MB * 4][64], const GemvArgs &p, int m0,
                                          int n0) {
    for (int i = threadIdx.x; i < MB * 256; i += kGemvWaves * 64) {
        const int l = i & 63, q = i >> 6, r = q & 3, a = q >> 2;
        const int m = m0 + 16 * a + 4 * (l >> 4) + r, n = n0 + (l & 15);
        if (m >= p.M || n >= p.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int s = 0; s < kGemvWaves; ++s) v += red[s][q][l];
        if constexpr (OUT_BF16) {
            if (p.C) v += (float)((const __bf16 *)p.C)[(int64_t)m * p.ldc + n];
            ((__bf16 *)p.D)[(int64_t)m * p.ldd + n] = (__bf16)v;
        } else {
            if (p.C) v += ((const float *)p.C)[(int64_t)m * p.ldc + n];
            ((float *)p.D)[(int64_t)m * p.ldd + n] = v;
        }
    }
}

// One MFMA of 32 K: 8 weights (a word of codes) of each lane against its x.
template <bool FP16, int MB>
__device__ __forceinline__ void gemv_step(const u32x4 (&xf)[MB], uint32_t w, uint32_t code, bool direct,
                                          f32x4 (&acc)[MB]) {
    const float scale = __builtin_bit_cast(float, code << 23);
    if (!FP16 || direct) {
        const u32x4 wf = fp4_up<FP16>(w, scale);
#pragma unroll
        for (int a = 0; a < MB; ++a) acc[a] = mfma16<FP16>(xf[a], wf, acc[a]);
    } else {
        const u32x4 wf = fp4_up<false>(w, scale);
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            u32x4 hi, lo;
            split_f16(xf[a], hi, lo);
            acc[a] = mfma16<false>(hi, wf, acc[a]);
            acc[a] = mfma16<false>(lo, wf, acc[a]);
        }
    }
}

// fp16 holds a scaled weight exactly when its scale is 2^-23 .. 2^13
// (subnormals included).
__device__ __forceinline__ bool fp16_scale(uint32_t code) { return code >= 104u && code <= 140u; }

// Weight rows 16-byte aligned: each wave's K step of 512 (16 rows of 256
// bytes) goes straight to LDS in whole rows, sixteen lanes a row, and is
// read back a word per lane in the MFMA's own order, so that X is read in
// runs of 64 bytes and a step of 32 K has one scale.  Chunk c of row r sits
// at chunk c ^ r: the 16 rows of a read fall on all 64 banks.
template <bool FP16, bool OUT_BF16, int MB>
__global__ void __launch_bounds__(kGemvWaves * 64) gemv_mxfp4_staged_kernel(GemvArgs p) {
    __shared__ __attribute__((aligned(16))) char stage[kGemvWaves][4096];
    __shared__ float red[kGemvWaves][MB * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lc = lane & 15, lg = lane >> 4;
    const int tn = blockIdx.x % p.tiles_n, tm = blockIdx.x / p.tiles_n;
    const int n0 = tn * 16, m0 = tm * 16 * MB;
    const int K = p.K;
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(p.W + (int64_t)n0 * p.ldw_bytes, span_bytes(p.N - n0, K / 2, p.ldw_bytes, 1));
    char *ring = stage[wave];
    const int64_t srow = n0 + lc < p.N ? n0 + lc : p.N - 1;
    const uint8_t *sf = p.SF + srow * p.ldsf;
    const uint16_t *x[MB];
    bool xin[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const int m = m0 + 16 * a + lc;
        xin[a] = m < p.M;
        x[a] = (const uint16_t *)p.X + (int64_t)(xin[a] ? m : 0) * p.ldx + 8 * lg;
    }
    f32x4 acc[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int k0 = wave * 512; k0 < K; k0 += kGemvWaves * 512) {
        // four rows an instruction: lane L writes chunk L % 16 of row 4 i + L / 16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * i + lg, c = lc ^ row;
            const int kb = k0 / 2 + c * 16;            // (rows past N lie past the resource)
            dma_load<16>(rW, ring + i * 1024, kb < K / 2 ? (uint32_t)(row * p.ldw_bytes + kb) : kOOB);
        }
        // byte j of sc[t]: the scale of K block 4 t + j
        uint32_t sc[4];
        if (p.kshift == 5 && k0 + 512 <= K) {
            const u32x4 v = ((const Bytes16 *)(sf + k0 / 32))->v;
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[t] = v[t];
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                sc[t] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = k0 + t * 128 + j * 32;
                    sc[t] |= (k < K ? (uint32_t)sf[k >> p.kshift] : 127u) << (8 * j);
                }
            }
        }
        bool direct = true;
        if constexpr (FP16) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) direct = direct && fp16_scale((sc[t] >> (8 * j)) & 0xffu);
            direct = __all(direct);
        }
        u32x4 xf[4][MB];
        auto load_x = [&](int t, int j) __attribute__((always_inline)) {
            const int k = k0 + t * 128 + j * 32;
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                xf[j][a] = u32x4{0u, 0u, 0u, 0u};
                if (xin[a] && k < K) xf[j][a] = ((const Halves8 *)(x[a] + k))->v;
            }
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) load_x(0, j);
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (t > 0) load_x(t, j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = *(const uint32_t *)(ring + lc * 256 + (((4 * t + j) ^ lc) << 4) + 4 * lg);
                gemv_step<FP16, MB>(xf[j], w, (sc[t] >> (8 * j)) & 0xffu, direct, acc);
            }
        }
        wait_lgkmcnt0();                               // this step's reads done before the next overwrites it
        asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][a * 4 + r][lane] = acc[a][r];
    __syncthreads();
    gemv_join<OUT_BF16, MB>(red, p, m0, n0);
}

// Weight rows that start at any byte.
template <bool FP16, bool OUT_BF16, int MB>
__global__ void __launch_bounds__(kGemvWaves * 64) gemv_mxfp4_kernel(GemvArgs p) {
    __shared__ float red[kGemvWaves][MB * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lc = lane & 15, lg = lane >> 4;
    const int tn = blockIdx.x % p.tiles_n, tm = blockIdx.x / p.tiles_n;
    const int n0 = tn * 16, m0 = tm * 16 * MB;
    const int K = p.K;
    // (rows past N: the last row again, never stored)
    const int64_t wrow = n0 + lc < p.N ? n0 + lc : p.N - 1;
    const uint8_t *w = p.W + wrow * p.ldw_bytes, *sf = p.SF + wrow * p.ldsf;
    const uint16_t *x[MB];
    bool xin[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const int m = m0 + 16 * a + lc;
        xin[a] = m < p.M;
        x[a] = (const uint16_t *)p.X + (int64_t)(xin[a] ? m : 0) * p.ldx;
    }
    f32x4 acc[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // wave w takes the K steps of 512 w, w + 8, ...: four tiles of 128, of
    // which lane group g loads block g, K permuted inside the tile
    for (int64_t k0 = (int64_t)wave * 512; k0 < K; k0 += kGemvWaves * 512) {
        u32x4 wq[4];
        uint32_t code[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t k = k0 + t * 128 + lg * 32;
            wq[t] = u32x4{0u, 0u, 0u, 0u};
            code[t] = 127u;
            if (k < K) {
                wq[t] = ((const Bytes16 *)(w + k / 2))->v;
                code[t] = sf[k >> p.kshift];
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t k = k0 + t * 128 + lg * 32;
            const bool direct = !FP16 || __all(fp16_scale(code[t]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 xf[MB];
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    xf[a] = u32x4{0u, 0u, 0u, 0u};
                    if (xin[a] && k < K) xf[a] = ((const Halves8 *)(x[a] + k + 8 * j))->v;
                }
                gemv_step<FP16, MB>(xf, wq[t][j], code[t], direct, acc);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][a * 4 + r][lane] = acc[a][r];
    __syncthreads();
    gemv_join<OUT_BF16, MB>(red, p, m0, n0);
}

template <bool FP16, bool OUT_BF16, int MB>
hipError_t go_gemv(const GemvArgs &p, unsigned grid, hipStream_t s) {
    // 16-byte weight rows
    if (((uintptr_t)p.W | (uintptr_t)p.ldw_bytes) % 16 == 0)
        hipLaunchKernelGGL((gemv_mxfp4_staged_kernel<FP16, OUT_BF16, MB>), dim3(grid), dim3(kGemvWaves * 64), 0, s, p);
    else
        hipLaunchKernelGGL((gemv_mxfp4_kernel<FP16, OUT_BF16, MB>), dim3(grid), dim3(kGemvWaves * 64), 0, s, p);
    return hipGetLastError();
}

template <bool FP16, bool OUT_BF16>
hipError_t launch_gemv(const GemvArgs &p, unsigned grid, hipStream_t s) {
    return p.M > 16 ? go_gemv<FP16, OUT_BF16, 2>(p, grid, s) : go_gemv<FP16, OUT_BF16, 1>(p, grid, s);
}

}  // namespace tg

extern "C" {

gemm_status gemv_mxfp4(int64_t M, int64_t N, int64_t K, int64_t kblock, const void *X, int64_t ldx, int x_type,
                       const void *W, int64_t ldw, const void *SFW, int64_t ldsfw, const void *C, int64_t ldc, void *D,
                       int64_t ldd, int out_type, hipStream_t stream) {
    // (X's 2-byte alignment is checked below: W's rows may start at any byte)
    const Common a{M, N, K, X, ldx, W, ldw, C, ldc, D, ldd, out_type, 1};
    bool none = false;
    gemm_status st = validate(a, &none);
    if (st != GEMM_OK || none) return st;
    if (x_type != GEMM_TYPE_BF16 && x_type != GEMM_TYPE_FP16) return GEMM_ERR_UNSUPPORTED;
    if (K % 32 != 0 || kblock <= 0 || kblock % 32 != 0 || ldw % 2 != 0) return GEMM_ERR_UNSUPPORTED;
    int kshift = 31;                                   // one scale per row: every index is 0
    if (kblock < K) {
        if ((kblock & (kblock - 1)) != 0) return GEMM_ERR_UNSUPPORTED;
        kshift = __builtin_ctzll((uint64_t)kblock);
    }
    if (ldsfw < (K + kblock - 1) / kblock) return GEMM_ERR_BAD_LD;
    if (K > 0 && !SFW) return GEMM_ERR_NULL_POINTER;
    if (misaligned(X, 2)) return GEMM_ERR_MISALIGNED;
    const int64_t tn = (N + 15) / 16, tm = M > 16 ? (M + 31) / 32 : 1;
    if (tn * tm >= kMaxDim) return GEMM_ERR_UNSUPPORTED;
    tg::GemvArgs p;
    p.X = X;
    p.W = (const uint8_t *)W;
    p.SF = (const uint8_t *)SFW;
    p.C = C;
    p.D = D;
    p.ldx = ldx;
    p.ldw_bytes = ldw / 2;
    p.ldsf = ldsfw;
    p.ldc = ldc;
    p.ldd = ldd;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.kshift = kshift;
    p.tiles_n = (int)tn;
    const unsigned grid = (unsigned)(tn * tm);
    const bool b = out_type == GEMM_OUT_BF16;
    hipError_t e;
    if (x_type == GEMM_TYPE_FP16)
        e = b ? tg::launch_gemv<true, true>(p, grid, stream) : tg::launch_gemv<true, false>(p, grid, stream);
    else
        e = b ? tg::launch_gemv<false, true>(p, grid, stream) : tg::launch_gemv<false, false>(p, grid, stream);
    return launched(e);
}

}  // extern "C"
