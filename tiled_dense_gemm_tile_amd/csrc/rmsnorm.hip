// C ABI and kernels of the forward row operators: mxfp8_quantize, rmsnorm,
// rmsnorm_mxfp8 (include/tilegemm_ops.h).
//
// One pass: a row's elements stay in registers between the sum of squares
// and the output, so every element is read and written once and the bound is
// the HBM rate.  h is rounded to the row type before the sum because that
// stored h is what the backward pass and the next layer read.  The sum and
// rstd are fp64; y is formed in fp32 as (h * w) * rstd -- for 16-bit h and w
// the first product is exact -- and rounded once.  Codes of block-scaled rows
// are those of the y before any rounding: one code that fp32 tips over a
// border is off by up to an eighth of its value, and some thirty of 16384 x
// 4096 were, for 0.3 us where rows are few (256 x 4096 3.5 against 3.7 us) and
// nothing where they are many.  16384 x 4096 bf16 with residual to
// block-scaled rows 82 us (5.8 TB/s), one row 2.7 us (an empty launch: 1.6);
// 16384 x 14336 bf16 quantised 125 us (5.7 TB/s).
#include <math.h>

#include "rows.hpp"
#include "rows_api.hpp"

using namespace tg_api;

namespace tg {

struct NormArgs {
    const void *X, *R, *W;
    void *H, *Y;                                       // Y: the row type, or e4m3 codes
    uint8_t *SF;
    float *rstd;
    int64_t ldx, ldr, ldh, ldy, ldsf;
    int64_t rows, row0;                                // row0: the launch's first row
    int N;
    double eps, inv_n;
    bool w_f32;
};

// 1 / sqrt(ss / N + eps) to about 2^-46: the hardware's estimate and a Newton
// step.  A sum past fp32 gives 0.
__device__ __forceinline__ double row_rstd(const NormArgs &p, double ss) {
    const double x = __builtin_fma(ss, p.inv_n, p.eps);
    if (ss > 0x1.fffffep127) return 0.0;
    const double r = __builtin_amdgcn_rsq(x);
    return x > 0.0 ? __builtin_fma(0.5 * r, __builtin_fma(-x * r, r, 1.0), r) : r;
}

// VE elements of a normed row as block-scaled ones.  In fp32 y is off by 3 of
// its half steps of 2^-24 (rstd and two products rounded), so codes and scales
// that 8 of them up or down do not change are those of the exact y.  Where
// they do -- in one wave of some 200 -- the wave takes them from y in 64 bits,
// which also settles blocks with an infinity.
template <int T>
__device__ __forceinline__ void norm_mx_store(const typename RowVec<T>::V &h, const float (&w)[kVE<T>], double rstd,
                                              uint8_t *q, uint8_t *sf, int c) {
    constexpr int VE = kVE<T>;
    constexpr float UP = 1.0f + 0x1p-21f, DOWN = 1.0f - 0x1p-21f;
    const float rstd32 = (float)rstd;
    float y[VE], m = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        y[i] = Elem<T>::up(h[i]) * w[i] * rstd32;
        m = __builtin_fmaxf(m, __builtin_fabsf(y[i]));
    }
    auto join = [](auto &v, auto other) __attribute__((always_inline)) { v = v > other ? v : other; };
    uint32_t mb = __builtin_bit_cast(uint32_t, m);
    join(mb, dpp<kXor1>(mb));
    join(mb, dpp<kXor2>(mb));
    if constexpr (VE == 4) join(mb, dpp<kMirror8>(mb));
    m = __builtin_bit_cast(float, mb);
    uint32_t code = mx_code(__builtin_bit_cast(uint32_t, m * UP));
    const float inv = mx_inverse(code);
    struct __attribute__((packed, aligned(1))) Words {
        uint32_t w[VE / 4];
    } out;
    bool near = code != mx_code(__builtin_bit_cast(uint32_t, m * DOWN)) || !(m < __builtin_inff());
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
        uint32_t o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float by = inv * (k ? DOWN : UP);
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[i] * by, y[i + 1] * by, 0, false);
            o[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[i + 2] * by, y[i + 3] * by, v, true);
        }
        out.w[i / 4] = o[0];
        near = near || o[0] != o[1];
    }
    if (__any(near)) {
        // (h anew: 64-bit forms kept from the sum of squares on would not fit the registers)
        u32x4 hb = __builtin_bit_cast(u32x4, h);
        asm volatile("" : "+v"(hb));
        const typename RowVec<T>::V hv = __builtin_bit_cast(typename RowVec<T>::V, hb);
        auto exact = [&](int i) __attribute__((always_inline)) { return (double)Elem<T>::up(hv[i]) * (double)w[i] * rstd; };
        double top = 0.0;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const double a = __builtin_fabs(exact(i));
            if (a < 0x1.ffffffp127) join(top, a);     // (what fp32 holds; no NaN)
        }
        join(top, dpp64<kXor1>(top));
        join(top, dpp64<kXor2>(top));
        if constexpr (VE == 4) join(top, dpp64<kMirror8>(top));
        // mx_code of a double: the exponent field is e + 8 + 1023
        const uint32_t f = (uint32_t)((__builtin_bit_cast(uint64_t, top) + ((1ull << 50) - 1)) >> 52);
        code = f > 904u ? f - 904u : 0u;
        const double by = __builtin_bit_cast(double, (uint64_t)(1150u - code) << 52);
        float v[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            // (cut to 24 bits with the last one telling of what was cut, which
            // the rounding to a code then sees)
            const double d = exact(i);
            uint64_t b = __builtin_bit_cast(uint64_t, d * by);
            b = (b & ~0x1fffffffull) | ((b & 0x1fffffffull) ? 1ull << 29 : 0);
            v[i] = __builtin_fabs(d) < 0x1.ffffffp127 ? (float)__builtin_bit_cast(double, b) : __builtin_nanf("");
        }
#pragma unroll
        for (int i = 0; i < VE; i += 4) {
            int o = __builtin_amdgcn_cvt_pk_fp8_f32(v[i], v[i + 1], 0, false);
            out.w[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[i + 2], v[i + 3], o, true);
        }
    }
    *(Words *)(q + c) = out;
    if (c % 32 == 0) sf[c / 32] = (uint8_t)code;
}

// TPR threads per row (64 or 128: four or two rows per workgroup of 256; 256
// or 1024: the workgroup), VPT vectors of 16 bytes per thread: N <= TPR * VPT *
// VE.
template <int T, bool MX, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rmsnorm_kernel(NormArgs p) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE, RPB = TPR < 256 ? 256 / TPR : 1;
    const int t = threadIdx.x % TPR;
    const int64_t row = p.row0 + (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (TPR == 64 && row >= p.rows) return;
    const bool in = TPR != 128 || row < p.rows;        // (rows of two waves meet at a barrier)
    const int N = p.N;
    const typename RV::S *x = (const typename RV::S *)p.X + row * p.ldx;
    const typename RV::S *r = (const typename RV::S *)p.R + row * p.ldr;

    typename RV::V h[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * VE;
        h[i] = typename RV::V{};
        if (in && c < N) h[i] = MX ? RV::load_whole(x, c) : RV::load_raw(x, c, N);
    }
    if (p.R) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * VE;
            if (in && c < N) {
                const typename RV::V v = MX ? RV::load_whole(r, c) : RV::load_raw(r, c, N);
#pragma unroll
                for (int u = 0; u < VE; ++u)
                    h[i][u] = Elem<T>::down(Elem<T>::up(h[i][u]) + Elem<T>::up(v[u]));
            }
        }
    }
    if constexpr (!MX) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * VE;
            if (c < N) h[i] = RV::settle(h[i], c, N);
        }
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int u = 0; u < VE; ++u) {
            const double f = (double)Elem<T>::up(h[i][u]);
            ss = __builtin_fma(f, f, ss);
        }
    ss = wave_sum64(ss);
    if constexpr (TPR > 64) {
        __shared__ double part[RPB][TPR / 64];
        if ((t & 63) == 0) part[threadIdx.x / TPR][t >> 6] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) ss += part[threadIdx.x / TPR][w];
    }
    const double rstd = row_rstd(p, ss);
    if (in && p.rstd && t == 0) p.rstd[row] = (float)rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * VE;
        if (in && c < N) {
            float w[VE];
            if constexpr (MX) {
                if (p.H) RV::store_whole((typename RV::S *)p.H + row * p.ldh, c, h[i]);
                load_weights<T, true>(p.W, p.w_f32, c, N, w);
                norm_mx_store<T>(h[i], w, rstd, (uint8_t *)p.Y + row * p.ldy, p.SF + row * p.ldsf, c);
            } else {
                if (p.H) RV::store((typename RV::S *)p.H + row * p.ldh, c, N, h[i]);
                load_weights<T>(p.W, p.w_f32, c, N, w);
                typename RV::V o;
#pragma unroll
                for (int u = 0; u < VE; ++u) o[u] = Elem<T>::down(Elem<T>::up(h[i][u]) * w[u] * (float)rstd);
                RV::store((typename RV::S *)p.Y + row * p.ldy, c, N, o);
            }
        }
    }
}

// Rows too long for the registers of one workgroup: two passes, the second
// reading the row again (h from H where it was written, else x + r again).
template <int T, bool MX>
__device__ __forceinline__ void rmsnorm_long_row(const NormArgs &p, int64_t row) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE;
    const int N = p.N, t = threadIdx.x;
    const typename RV::S *x = (const typename RV::S *)p.X + row * p.ldx;
    const typename RV::S *r = (const typename RV::S *)p.R + row * p.ldr;
    typename RV::S *hs = (typename RV::S *)p.H + row * p.ldh;
    auto sum_at = [&](int64_t c) __attribute__((always_inline)) {
        typename RV::V h = RV::load(x, (int)c, N);
        if (p.R) {
            const typename RV::V v = RV::load(r, (int)c, N);
#pragma unroll
            for (int u = 0; u < VE; ++u) h[u] = Elem<T>::down(Elem<T>::up(h[u]) + Elem<T>::up(v[u]));
        }
        return h;
    };
    double ss = 0.0;
    for (int64_t c = (int64_t)t * VE; c < N; c += 1024 * VE) {
        const typename RV::V h = sum_at(c);
#pragma unroll
        for (int u = 0; u < VE; ++u) {
            const double f = (double)Elem<T>::up(h[u]);
            ss = __builtin_fma(f, f, ss);
        }
        if (p.H) RV::store(hs, (int)c, N, h);
    }
    __shared__ double part[16];
    ss = wave_sum64(ss);
    if ((t & 63) == 0) part[t >> 6] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) ss += part[w];
    const double rstd = row_rstd(p, ss);
    if (p.rstd && t == 0) p.rstd[row] = (float)rstd;
    for (int64_t c = (int64_t)t * VE; c < N; c += 1024 * VE) {
        const typename RV::V h = p.H ? RV::load(hs, (int)c, N) : sum_at(c);   // this thread's own stores
        float w[VE];
        load_weights<T>(p.W, p.w_f32, (int)c, N, w);
        if constexpr (MX) {
            norm_mx_store<T>(h, w, rstd, (uint8_t *)p.Y + row * p.ldy, p.SF + row * p.ldsf, (int)c);
        } else {
            typename RV::V o;
#pragma unroll
            for (int u = 0; u < VE; ++u) o[u] = Elem<T>::down(Elem<T>::up(h[u]) * w[u] * (float)rstd);
            RV::store((typename RV::S *)p.Y + row * p.ldy, (int)c, N, o);
        }
    }
}

template <int T, bool MX>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(NormArgs p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        rmsnorm_long_row<T, MX>(p, row);
        __syncthreads();                               // (the row's sums in LDS)
    }
}

// One vector of one row per thread and step; blocks of 32 elements are
// independent, so rows need no workgroup of their own.  STREAM: codes are
// stored past the caches, for results larger than the memory-side cache holds
// for the next reader (16384 x 14336 bf16: 123.6 against 129.6 us).
template <int T, bool STREAM>
__global__ void __launch_bounds__(256)
    quantize_kernel(const void *X, int64_t ldx, uint8_t *Q, int64_t ldq, uint8_t *SF, int64_t ldsf, int64_t rows,
                    int nvec) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE;
    const int64_t total = rows * nvec;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / nvec;
        const int c = (int)(i - row * nvec) * VE;
        const typename RV::V v = RV::load((const typename RV::S *)X + row * ldx, c, c + VE);
        float y[VE];
#pragma unroll
        for (int u = 0; u < VE; ++u) y[u] = Elem<T>::up(v[u]);
        mx_store<VE, STREAM>(y, Q + row * ldq, SF + row * ldsf, c);
    }
}

template <int T, bool MX, int TPR, int VPT>
hipError_t go(NormArgs &p, hipStream_t s) {
    constexpr int rows = TPR < 256 ? 256 / TPR : 1;
    hipError_t e = hipSuccess;
    for (p.row0 = 0; p.row0 < p.rows && e == hipSuccess; p.row0 += kMaxGrid * rows) {
        const int64_t blocks = (p.rows - p.row0 + rows - 1) / rows;
        hipLaunchKernelGGL((rmsnorm_kernel<T, MX, TPR, VPT>), dim3((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid)),
                           dim3(TPR < 256 ? 256 : TPR), 0, s, p);
        e = hipGetLastError();
    }
    return e;
}

template <int T, bool MX>
hipError_t launch_norm(NormArgs &p, hipStream_t s) {
    const int nvec = (int)(((int64_t)p.N + kVE<T> - 1) / kVE<T>);
    // The fewest vectors per thread: a row's loads are all in flight at once
    // either way, and more waves share a row's arithmetic (16384 x 4096 bf16
    // with residual to mxfp8: 84 us with 256 threads of two vectors, 82 with
    // 512 of one; 107 with a wave of eight).
    if (nvec <= 64) return go<T, MX, 64, 1>(p, s);
    if (nvec <= 128) return go<T, MX, 128, 1>(p, s);
    if (nvec <= 256) return go<T, MX, 256, 1>(p, s);
    // 512 threads where three quarters of them have work (8192 x 8192 bf16 84.7
    // against 91.4, one row 3.3 against 4.4; 16384 x 2304 59.9 against 52.1)
    // and two loads each (16384 x 3968 without residual 44.0 against 35.2).  The
    // count of rows plays no part: a row's bits do not depend on its batch.
    if (nvec <= 384 || (nvec <= 512 && !p.R)) return go<T, MX, 256, 2>(p, s);
    if (nvec <= 512) return go<T, MX, 512, 1>(p, s);
    if (nvec <= 768) return go<T, MX, 256, 4>(p, s);
    if (nvec <= 1024) return go<T, MX, 512, 2>(p, s);
    if (nvec <= 2048) return go<T, MX, 512, 4>(p, s);
    if (nvec <= 4096) return go<T, MX, 1024, 4>(p, s);
    hipLaunchKernelGGL((rmsnorm_long_kernel<T, MX>), dim3((unsigned)(p.rows < 2048 ? p.rows : 2048)), dim3(1024),
                       0, s, p);
    return hipGetLastError();
}

}  // namespace tg

namespace {

gemm_status run_norm(bool mx, int64_t rows, int64_t N, const void *X, int64_t ldx, const void *R, int64_t ldr,
                     int type, const void *W, int w_type, float eps, void *H, int64_t ldh, void *Y, int64_t ldy,
                     void *SF, int64_t ldsf, float *rstd, hipStream_t s) {
    bool none;
    gemm_status st = check_rows(rows, N, &none);
    if (st != GEMM_OK) return st;
    if (!elem_type(type) || (w_type != type && w_type != GEMM_TYPE_F32)) return GEMM_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || !isfinite(eps) || (mx && N % 32 != 0)) return GEMM_ERR_UNSUPPORTED;
    if (none) return GEMM_OK;
    if (ldx < N || (R && ldr < N) || (H && ldh < N) || ldy < N || (mx && ldsf < N / 32)) return GEMM_ERR_BAD_LD;
    if (!X || !W || !Y || (mx && !SF)) return GEMM_ERR_NULL_POINTER;
    const int es = elem_size(type);
    if (misaligned(X, es) || misaligned(R, es) || misaligned(H, es) || misaligned(Y, mx ? 1 : es) ||
        misaligned(W, elem_size(w_type)) || misaligned(rstd, 4))
        return GEMM_ERR_MISALIGNED;
    if ((H && H == Y) || (H == X && ldh != ldx) || (H && H == R && ldh != ldr)) return GEMM_ERR_UNSUPPORTED;
    if ((Y == X && ldy != ldx) || (Y == R && ldy != ldr) || (mx && (Y == X || Y == R || Y == SF))) return GEMM_ERR_UNSUPPORTED;
    tg::NormArgs p;
    p.X = X;
    p.R = R;
    p.W = W;
    p.H = H;
    p.Y = Y;
    p.SF = (uint8_t *)SF;
    p.rstd = rstd;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.ldy = ldy;
    p.ldsf = ldsf;
    p.rows = rows;
    p.N = (int)N;
    p.eps = eps;
    p.inv_n = 1.0 / (double)N;
    p.w_f32 = w_type == GEMM_TYPE_F32;
    hipError_t e;
    switch (type) {
    case GEMM_TYPE_F32: e = mx ? tg::launch_norm<0, true>(p, s) : tg::launch_norm<0, false>(p, s); break;
    case GEMM_TYPE_BF16: e = mx ? tg::launch_norm<1, true>(p, s) : tg::launch_norm<1, false>(p, s); break;
    default: e = mx ? tg::launch_norm<2, true>(p, s) : tg::launch_norm<2, false>(p, s); break;
    }
    return launched(e);
}

}  // namespace

extern "C" {

gemm_status rmsnorm(int64_t rows, int64_t N, const void *X, int64_t ldx, const void *R, int64_t ldr, int type,
                    const void *W, int w_type, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, float *rstd,
                    hipStream_t stream) {
    return run_norm(false, rows, N, X, ldx, R, ldr, type, W, w_type, eps, H, ldh, Y, ldy, nullptr, 0, rstd, stream);
}

gemm_status rmsnorm_mxfp8(int64_t rows, int64_t N, const void *X, int64_t ldx, const void *R, int64_t ldr, int type,
                          const void *W, int w_type, float eps, void *H, int64_t ldh, void *Q, int64_t ldq, void *SF,
                          int64_t ldsf, float *rstd, hipStream_t stream) {
    return run_norm(true, rows, N, X, ldx, R, ldr, type, W, w_type, eps, H, ldh, Q, ldq, SF, ldsf, rstd, stream);
}

gemm_status mxfp8_quantize(int64_t rows, int64_t N, const void *X, int64_t ldx, int x_type, void *Q, int64_t ldq,
                           void *SF, int64_t ldsf, hipStream_t stream) {
    bool none;
    gemm_status st = check_rows(rows, N, &none);
    if (st != GEMM_OK) return st;
    if (!elem_type(x_type) || N % 32 != 0) return GEMM_ERR_UNSUPPORTED;
    if (none) return GEMM_OK;
    if (ldx < N || ldq < N || ldsf < N / 32) return GEMM_ERR_BAD_LD;
    if (!X || !Q || !SF) return GEMM_ERR_NULL_POINTER;
    if (misaligned(X, elem_size(x_type))) return GEMM_ERR_MISALIGNED;
    if (Q == X || SF == X || SF == Q) return GEMM_ERR_UNSUPPORTED;
    const int ve = x_type == GEMM_TYPE_F32 ? 4 : 8;
    const int nvec = (int)(N / ve);
    const int64_t want = (rows * nvec + 255) / 256;
    const unsigned grid = (unsigned)(want < 16384 ? want : 16384);
    switch (x_type) {
#define TG_QUANT(t)                                                                                                  \
    if (rows * N >= (int64_t)128 << 20)                                                                              \
        hipLaunchKernelGGL((tg::quantize_kernel<t, true>), dim3(grid), dim3(256), 0, stream, X, ldx, (uint8_t *)Q,   \
                           ldq, (uint8_t *)SF, ldsf, rows, nvec);                                                    \
    else                                                                                                             \
        hipLaunchKernelGGL((tg::quantize_kernel<t, false>), dim3(grid), dim3(256), 0, stream, X, ldx, (uint8_t *)Q,  \
                           ldq, (uint8_t *)SF, ldsf, rows, nvec)
    case GEMM_TYPE_F32: TG_QUANT(0); break;
    case GEMM_TYPE_BF16: TG_QUANT(1); break;
    default: TG_QUANT(2); break;
#undef TG_QUANT
    }
    return launched(hipGetLastError());
}

}  // extern "C"
