// C ABI of gemm_int8 and int8_quantize (include/tilegemm_layers.h), and the
// quantisation's kernels.
#include "prod_api.hpp"

using namespace tg_api;

namespace tg {

// One row in the registers of NT threads, NV vectors of 16 bytes each; WIDE
// rows are read twice (the second time from the caches).  The row's largest
// magnitude as bits: an infinity or a NaN shows as a larger number than any
// finite one.  Bound by memory (8192 x 14336 bf16 66 to 75 us, 4.7 to 5.3 TB/s).
struct QuantArgs {
    const void *X;
    int8_t *Q;
    float *S;
    int64_t ldx, ldq, rows;
    int N;
};

// x / s rounded to nearest even, exactly: x * (1 / s) is off by 2^-16 at most
// (three roundings of a number up to 127), so only within 2^-14 of a border the
// remainder's sign decides.  It is a multiple of half of s's last place, so both
// are scaled up first where that may be below the least subnormal, 2^-149.
__device__ __forceinline__ int int8_code(float x, float s, float inv) {
    const float y = x * inv;
    float r = rintf(y);
    if (fabsf(y - r) > 0.5f - 0x1p-14f) {
        const float up = s < 1.0f ? 0x1p24f : 1.0f;
        const float h = floorf(y) + 0.5f, d = fmaf(-h, s * up, x * up);
        r = d > 0.0f ? h + 0.5f : d < 0.0f ? h - 0.5f : rintf(h);
    }
    return (int)r;
}

template <int T, int VE>
__device__ __forceinline__ uint32_t magnitude(const typename RowVec<T>::V &v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, Elem<T>::up(v[i])) & 0x7fffffffu;
        m = m > b ? m : b;
    }
    return m;
}

template <int T>
__device__ __forceinline__ void store_codes(int8_t *q, int c, int n, const typename RowVec<T>::V &v, bool finite,
                                            float s, float inv) {
    constexpr int VE = kVE<T>;
    struct __attribute__((packed, aligned(1))) Words {
        uint32_t w[VE / 4];
    } o;
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w |= ((uint32_t)int8_code(finite ? Elem<T>::up(v[i + k]) : 0.0f, s, inv) & 255u) << (8 * k);
        o.w[i / 4] = w;
    }
    if (c + VE <= n) {
        *(Words *)(q + c) = o;
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (c + i < n) q[c + i] = (int8_t)(o.w[i / 4] >> (8 * (i % 4)));
    }
}

template <int T, int NT, int NV, bool WIDE>
__global__ void __launch_bounds__(NT < 128 ? 256 : NT) int8_quantize_kernel(QuantArgs p) {
    constexpr int VE = kVE<T>, RPW = NT < 128 ? 256 / NT : 1, NW = NT / 64;    // rows of a workgroup, waves of a row
    const int t = threadIdx.x % NT, sub = threadIdx.x / NT;
    const int lane = threadIdx.x & 63, wave = t >> 6;
    __shared__ uint32_t top[NW > 1 ? NW : 1];
    for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < p.rows; row += (int64_t)gridDim.x * RPW) {
        const void *x = (const typename RowVec<T>::S *)p.X + row * p.ldx;
        typename RowVec<T>::V v[WIDE ? 1 : NV];
        uint32_t m = 0;
        if constexpr (WIDE) {
            for (int c = t * VE; c < p.N; c += NT * VE) {
                const uint32_t b = magnitude<T, VE>(RowVec<T>::load(x, c, p.N));
                m = m > b ? m : b;
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * NT + t) * VE;
                v[k] = {};
                if (c < p.N) v[k] = RowVec<T>::load_raw(x, c, p.N);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * NT + t) * VE;
                if (c < p.N) v[k] = RowVec<T>::settle(v[k], c, p.N);
                const uint32_t b = magnitude<T, VE>(v[k]);
                m = m > b ? m : b;
            }
        }
        auto join = [&](uint32_t b) __attribute__((always_inline)) { m = m > b ? m : b; };
        join(dpp<kXor1>(m));
        join(dpp<kXor2>(m));
        join(dpp<kMirror8>(m));
        join(dpp<kMirror16>(m));
        join(__shfl_xor(m, 16));
        join(__shfl_xor(m, 32));
        if constexpr (NW > 1) {
            __syncthreads();                           // (the last row's reads of top)
            if (lane == 0) top[wave] = m;
            __syncthreads();
            m = top[0];
#pragma unroll
            for (int k = 1; k < NW; ++k) m = m > top[k] ? m : top[k];
        }
        const bool finite = m < 0x7f800000u;
        const float s = finite ? fmaxf(__builtin_bit_cast(float, m) / 127.0f, 0x1p-126f)
                               : __builtin_bit_cast(float, 0x7fc00000u);
        const float inv = 1.0f / s;
        int8_t *q = p.Q + row * p.ldq;
        if (t == 0) p.S[row] = s;
        if constexpr (WIDE) {
            for (int c = t * VE; c < p.N; c += NT * VE)
                store_codes<T>(q, c, p.N, RowVec<T>::load(x, c, p.N), finite, s, inv);
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * NT + t) * VE;
                if (c < p.N) store_codes<T>(q, c, p.N, v[k], finite, s, inv);
            }
        }
    }
}

template <int T, int NT, int NV, bool WIDE = false>
hipError_t go_quantize(const QuantArgs &p, hipStream_t s) {
    constexpr int RPW = NT < 128 ? 256 / NT : 1;
    const int64_t want = (p.rows + RPW - 1) / RPW;
    hipLaunchKernelGGL((int8_quantize_kernel<T, NT, NV, WIDE>), dim3((unsigned)(want < kMaxGrid ? want : kMaxGrid)),
                       dim3(NT < 128 ? 256 : NT), 0, s, p);
    return hipGetLastError();
}

template <int T>
hipError_t launch_quantize(const QuantArgs &p, hipStream_t s) {
    const int nvec = (int)(((int64_t)p.N + kVE<T> - 1) / kVE<T>);
    if (nvec <= 64) return go_quantize<T, 64, 1>(p, s);
    // Few rows: as many threads as there are vectors (64 x 14336 bf16: 4.9 us, of
    // 256 threads 8.1).  Many: more vectors a thread, as joining the threads'
    // maxima and the division come once a row (16384 x 4096 bf16: 256 x 2 37.3,
    // 512 x 1 58.5; 20000 x 1024: 64 x 2 14.1, 128 x 1 18.9, 256 x 1 28.2; 8192
    // x 2048: 128 x 2 12.9, 256 x 1 16.4).
    if (p.rows < 1024) {
        if (nvec <= 128) return go_quantize<T, 128, 1>(p, s);
        if (nvec <= 256) return go_quantize<T, 256, 1>(p, s);
        if (nvec <= 512) return go_quantize<T, 512, 1>(p, s);
        if (nvec <= 1024) return go_quantize<T, 1024, 1>(p, s);
        if (nvec <= 2048) return go_quantize<T, 1024, 2>(p, s);
    } else {
        if (nvec <= 128) return go_quantize<T, 64, 2>(p, s);
        if (nvec <= 256) return go_quantize<T, 128, 2>(p, s);
        if (nvec <= 512) return go_quantize<T, 256, 2>(p, s);
        if (nvec <= 1024) return go_quantize<T, 256, 4>(p, s);
        if (nvec <= 2048) return go_quantize<T, 256, 8>(p, s);
    }
    if (nvec <= 4096) return go_quantize<T, 512, 8>(p, s);
    return go_quantize<T, 1024, 1, true>(p, s);
}

}  // namespace tg

extern "C" {

gemm_status int8_quantize(int64_t rows, int64_t N, const void *X, int64_t ldx, int x_type, void *Q, int64_t ldq,
                          float *S, hipStream_t stream) {
    bool none;
    gemm_status st = check_rows(rows, N, &none);
    if (st != GEMM_OK) return st;
    if (!elem_type(x_type)) return GEMM_ERR_UNSUPPORTED;
    if (rows == 0) return GEMM_OK;
    if (ldx < N || ldq < N) return GEMM_ERR_BAD_LD;
    if (!S || (N > 0 && (!X || !Q))) return GEMM_ERR_NULL_POINTER;
    const int es = elem_size(x_type);
    if (misaligned(X, es) || misaligned(S, 4)) return GEMM_ERR_MISALIGNED;
    if (N > 0 && (overlap(Q, matrix_bytes(rows, N, ldq, 1), X, matrix_bytes(rows, N, ldx, es)) ||
                  overlap(S, rows * 4, X, matrix_bytes(rows, N, ldx, es)) ||
                  overlap(S, rows * 4, Q, matrix_bytes(rows, N, ldq, 1))))
        return GEMM_ERR_UNSUPPORTED;
    const tg::QuantArgs p{X, (int8_t *)Q, S, ldx, ldq, rows, (int)N};
    switch (x_type) {
    case GEMM_TYPE_F32: return launched(tg::launch_quantize<0>(p, stream));
    case GEMM_TYPE_BF16: return launched(tg::launch_quantize<1>(p, stream));
    default: return launched(tg::launch_quantize<2>(p, stream));
    }
}

size_t gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M >= kMostRows || N >= kMostRows || K >= (int64_t)1 << 17) return 0;
    return prod_copy_bytes(M, N, 1, K);
}

gemm_status gemm_int8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const float *SA, const void *B,
                      int64_t ldb, const float *SB, const void *C, int64_t ldc, void *D, int64_t ldd, int out_type,
                      void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_SIZE;
    if (M >= kMostRows || N >= kMostRows || K >= (int64_t)1 << 17 || !elem_type(out_type)) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (lda < K || ldb < K || ldd < N || (C && ldc != 0 && ldc < N)) return GEMM_ERR_BAD_LD;
    if (!D || !SA || !SB || (K > 0 && (!A || !B))) return GEMM_ERR_NULL_POINTER;
    const int os = elem_size(out_type);
    if (misaligned(SA, 4) || misaligned(SB, 4) || misaligned(C, os) || misaligned(D, os)) return GEMM_ERR_MISALIGNED;
    if (lda >= kMaxLdBytes || ldb >= kMaxLdBytes || ldd * os >= kMaxLdBytes || (C && ldc * os >= kMaxLdBytes))
        return GEMM_ERR_UNSUPPORTED;
    const Area d{D, M, N, ldd, os}, in[5] = {{A, M, K, lda, 1}, {B, N, K, ldb, 1}, {SA, 1, M, M, 4}, {SB, 1, N, N, 4},
                                             {C, ldc ? M : 1, N, ldc ? ldc : N, os}};
    if (C && C == D && ldc != ldd && M > 1) return GEMM_ERR_UNSUPPORTED;
    for (int i = 0; i < (C == D ? 4 : 5); ++i)
        if (near(d, in[i])) return GEMM_ERR_UNSUPPORTED;
    if (workspace && (uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
    tg::ProdArgs p = {};
    p.A = A;
    p.B = B;
    p.lda = lda;
    p.ldb = ldb;
    p.M = (int)M;
    p.N = (int)N;
    p.KB = (int)K;
    const size_t need = workspace && !prod_aligned(p) ? prod_copy_bytes(M, N, 1, K) : 0;
    if (need > 0 && workspace_bytes >= need) {
        if (near(d, workspace, need)) return GEMM_ERR_UNSUPPORTED;
        for (const Area &a : in)
            if (near(a, workspace, need)) return GEMM_ERR_UNSUPPORTED;
        gemm_status st = launched(tg::prod_aligned_copies(p, tg::kI8, (char *)workspace, stream));
        if (st != GEMM_OK) return st;
    }
    const bool vec = tg::emit_whole(D, ldd, N, os);
    switch (out_type) {
    case GEMM_TYPE_F32: return launched(tg::launch_int8<0>(p, {SA, SB, C, D, ldc, ldd, vec, C != nullptr}, stream));
    case GEMM_TYPE_BF16: return launched(tg::launch_int8<1>(p, {SA, SB, C, D, ldc, ldd, vec, C != nullptr}, stream));
    default: return launched(tg::launch_int8<2>(p, {SA, SB, C, D, ldc, ldd, vec, C != nullptr}, stream));
    }
}

}  // extern "C"
