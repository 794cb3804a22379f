// grad_norm and grad_clip (include/tilegemm_layers.h): the sum of all
// gradients' squares, and their scaling.
//
// Bound by memory: one read for the sum (1.3 G elements of bf16 460 us, 5.7
// TB/s), one read and write for the scaling (980 us, 5.4 TB/s), and by the
// launches where gradients are few.  A launch takes up to 128
// tensors in its arguments (so that nothing is copied to the GPU and a captured
// graph holds what it needs), cut into chunks of 32 KiB that a fixed
// number of workgroups walks; each keeps its sum in fp64 and writes one partial
// sum.  The scaling's workgroups add up to kGradGroups partial sums for
// themselves, which costs less than a launch between the two; more of them one
// workgroup adds for all (each workgroup of each launch for itself: 6000 tensors
// of 128 K bf16 3.4 ms, so 1.2).  The scaling walks the chunks from the last to
// the first: the last ones read are still in the caches.
#include <algorithm>
#include <cstdlib>
#include <initializer_list>
#include <memory>

#include "rows_api.hpp"
#include "rows.hpp"

#include "../../include/tilegemm_layers.h"

using namespace tg_api;

namespace tg {

constexpr int kGradTable = 128, kGradFew = 16, kGradGroups = 2048;
// Elements of a chunk: 32 KiB, 8 vectors of each of 256 threads (half of that:
// 16-bit sums at 5.3 TB/s in place of 6.0).
template <int T> constexpr int kGradChunk = 8 * 256 * kVE<T>;

template <int MOST>
struct GradTable {
    const void *src[MOST];
    void *dst[MOST];
    int64_t n[MOST];
    uint32_t first[MOST + 1];                          // first chunk of each tensor; [count]: all chunks
    uint8_t type[MOST];
    int count;
};
static_assert(sizeof(GradTable<kGradTable>) <= 3800, "kernel arguments");

// The tensor whose chunk c is.
template <int MOST>
__device__ __forceinline__ int grad_tensor(const GradTable<MOST> &t, uint32_t c) {
    int lo = 0, hi = t.count;                          // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= c) lo = mid; else hi = mid;
    }
    return lo;
}

// f(vector, where, end) for each 16-byte vector of a chunk that is this
// thread's: a whole chunk's loads are all in flight at once, a tensor's last
// chunk goes vector by vector.
template <int T, class F>
__device__ __forceinline__ void grad_vectors(const void *src, uint32_t chunk, int64_t n, F &&f) {
    typedef RowVec<T> R;
    const int64_t begin = (int64_t)chunk * kGradChunk<T>;
    const typename R::S *p = (const typename R::S *)src + begin;
    constexpr int VE = R::VE, NV = 8;
    if (n - begin >= kGradChunk<T>) {
        typename R::V v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = R::load_whole(p, (k * 256 + (int)threadIdx.x) * VE);
#pragma unroll
        for (int k = 0; k < NV; ++k) f(v[k], (k * 256 + (int)threadIdx.x) * VE, kGradChunk<T>);
    } else {
        const int len = (int)(n - begin);
#pragma unroll 1
        for (int c = (int)threadIdx.x * VE; c < len; c += 256 * VE) f(R::load_each(p, c, len), c, len);
    }
}

__device__ __forceinline__ double group_sum(double v, double *lds) {
    v = wave_sum64(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

template <int MOST>
__global__ void __launch_bounds__(256) grad_squares_kernel(GradTable<MOST> t, double *part) {
    __shared__ double lds[4];
    double s[4] = {};                                  // (four chains of additions)
    const uint32_t chunks = t.first[t.count];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = __builtin_amdgcn_readfirstlane(grad_tensor(t, c));
        const uint32_t chunk = c - t.first[i];
        auto add = [&](auto type) __attribute__((always_inline)) {
            constexpr int T = decltype(type)::value;
            grad_vectors<T>(t.src[i], chunk, t.n[i], [&](auto v, int, int) __attribute__((always_inline)) {
#pragma unroll
                for (int k = 0; k < kVE<T>; ++k) {
                    const double d = (double)Elem<T>::up(v[k]);
                    s[k % 4] += d * d;
                }
            });
        };
        switch (t.type[i]) {
        case 0: add(std::integral_constant<int, 0>()); break;
        case 1: add(std::integral_constant<int, 1>()); break;
        default: add(std::integral_constant<int, 2>()); break;
        }
    }
    const double all = group_sum((s[0] + s[1]) + (s[2] + s[3]), lds);
    if (threadIdx.x == 0) part[blockIdx.x] = all;
}

// The norm from the partial sums, by one workgroup.
__device__ __forceinline__ float grad_total(const double *part, int parts, double *lds) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
    return (float)sqrt(group_sum(s, lds));
}

__global__ void __launch_bounds__(256) grad_norm_kernel(const double *part, int parts, float *norm) {
    __shared__ double lds[4];
    const float v = grad_total(part, parts, lds);
    if (threadIdx.x == 0) *norm = v;
}

template <int MOST>
__global__ void __launch_bounds__(256) grad_scale_kernel(GradTable<MOST> t, const double *part, int parts,
                                                         const float *given, float max_norm, float *norm, bool stream_out) {
    __shared__ double lds[4];
    const float v = given ? *given : grad_total(part, parts, lds);
    if (norm && norm != given && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float by = max_norm / (v + 1e-6f);
    by = by > 1.0f || (isinf(max_norm) && v == v) ? 1.0f : by;    // (a NaN stays one; inf / inf bounds nothing)
    const uint32_t chunks = t.first[t.count];
    for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
        const uint32_t c = chunks - 1 - k;
        const int i = __builtin_amdgcn_readfirstlane(grad_tensor(t, c));
        if (by == 1.0f && t.src[i] == t.dst[i]) continue;
        const uint32_t chunk = c - t.first[i];
        auto scale = [&](auto type) __attribute__((always_inline)) {
            constexpr int T = decltype(type)::value;
            typedef RowVec<T> R;
            typename R::S *to = (typename R::S *)t.dst[i] + (int64_t)chunk * kGradChunk<T>;
            grad_vectors<T>(t.src[i], chunk, t.n[i], [&](auto x, int at, int len) __attribute__((always_inline)) {
                typename R::V o;
#pragma unroll
                for (int j = 0; j < kVE<T>; ++j) o[j] = Elem<T>::down(Elem<T>::up(x[j]) * by);
                typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2)));
                if (stream_out && at + kVE<T> <= len)
                    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), (U *)(to + at));
                else
                    R::store(to, at, len, o);
            });
        };
        switch (t.type[i]) {
        case 0: scale(std::integral_constant<int, 0>()); break;
        case 1: scale(std::integral_constant<int, 1>()); break;
        default: scale(std::integral_constant<int, 2>()); break;
        }
    }
}

}  // namespace tg

namespace {

constexpr int64_t kMostGrads = (int64_t)1 << 20, kMostElements = (int64_t)1 << 40;

gemm_status check_grads(int64_t n, const void *const *src, void *const *dst, const int64_t *sizes, const int *types) {
    if (n < 0) return GEMM_ERR_INVALID_SIZE;
    if (n >= kMostGrads) return GEMM_ERR_UNSUPPORTED;
    if (n > 0 && (!src || !sizes || !types)) return GEMM_ERR_NULL_POINTER;
    int64_t all = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] < 0) return GEMM_ERR_INVALID_SIZE;
        if (sizes[i] >= kMostElements || !elem_type(types[i])) return GEMM_ERR_UNSUPPORTED;
        if (sizes[i] == 0) continue;
        if (!src[i] || (dst && !dst[i])) return GEMM_ERR_NULL_POINTER;
        if (misaligned(src[i], elem_size(types[i])) || (dst && misaligned(dst[i], elem_size(types[i]))))
            return GEMM_ERR_MISALIGNED;
        all += sizes[i];
        if (all >= kMostElements) return GEMM_ERR_UNSUPPORTED;
    }
    return GEMM_OK;
}

// Tensors [at, next) in one launch's table; a tensor of more chunks than a
// launch counts in 32 bits takes none (sizes below 2^40 have 2^27).
template <int MOST>
int64_t fill(tg::GradTable<MOST> &t, int64_t at, int64_t n, const void *const *src, void *const *dst, const int64_t *sizes,
             const int *types) {
    t.count = 0;
    t.first[0] = 0;
    for (; at < n && t.count < MOST; ++at) {
        if (sizes[at] == 0) continue;
        const int c = t.count++;
        t.src[c] = src[at];
        t.dst[c] = dst ? dst[at] : const_cast<void *>(src[at]);
        t.n[c] = sizes[at];
        t.type[c] = (uint8_t)types[at];
        const int64_t chunk = types[at] == GEMM_TYPE_F32 ? tg::kGradChunk<0> : tg::kGradChunk<1>;
        t.first[c + 1] = t.first[c] + (uint32_t)((sizes[at] + chunk - 1) / chunk);
    }
    return at;
}

template <int MOST>
unsigned groups(const tg::GradTable<MOST> &t) {
    const uint32_t c = t.first[t.count];
    return c < (uint32_t)tg::kGradGroups ? c : tg::kGradGroups;
}

// Partial sums of all tensors; *parts: how many.
template <int MOST>
gemm_status squares(int64_t n, const void *const *src, const int64_t *sizes, const int *types, double *part,
                    int *parts, hipStream_t s) {
    tg::GradTable<MOST> t;
    *parts = 0;
    for (int64_t at = 0; at < n;) {
        at = fill(t, at, n, src, nullptr, sizes, types);
        if (t.count == 0) break;
        const unsigned g = groups(t);
        hipLaunchKernelGGL(tg::grad_squares_kernel<MOST>, dim3(g), dim3(256), 0, s, t, part + *parts);
        const gemm_status st = launched(hipGetLastError());
        if (st != GEMM_OK) return st;
        *parts += (int)g;
    }
    return GEMM_OK;
}

// Whether a result shares memory with another one, with a gradient that is not
// its own, or with the call's other memory: results in the order of their
// addresses, then each piece looked up among them.  (What else is written:
// check_written.)
struct Span {
    uintptr_t from, to;
    int64_t i;
};
Span span_of(const void *p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes, 0}; }

gemm_status check_shared(int64_t n, const void *const *src, void *const *dst, const int64_t *sizes, const int *types,
                         std::initializer_list<Span> others) {
    constexpr int64_t kFew = 256;
    Span few[kFew];
    std::unique_ptr<Span, void (*)(void *)> many(nullptr, free);
    if (n > kFew) many.reset((Span *)malloc((size_t)n * sizeof(Span)));
    Span *const at = n > kFew ? many.get() : few;
    if (!at) return GEMM_ERR_UNSUPPORTED;
    int64_t count = 0;
    bool apart = false;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t from = (uintptr_t)(dst ? dst[i] : src[i]);
        at[count++] = {from, from + (uintptr_t)(sizes[i] * elem_size(types[i])), i};
        apart = apart || (dst && dst[i] != src[i]);
    }
    std::sort(at, at + count, [](const Span &a, const Span &b) { return a.from < b.from; });
    for (int64_t k = 1; k < count; ++k)
        if (at[k].from < at[k - 1].to) return GEMM_ERR_UNSUPPORTED;
    auto hit = [&](uintptr_t from, uintptr_t to) -> const Span * {
        const Span *s = std::lower_bound(at, at + count, to, [](const Span &a, uintptr_t v) { return a.from < v; });
        return s != at && s[-1].to > from ? s - 1 : nullptr;
    };
    for (int64_t i = 0; apart && i < n; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t from = (uintptr_t)src[i];
        const Span *s = hit(from, from + (uintptr_t)(sizes[i] * elem_size(types[i])));
        if (s && !(s->i == i && s->from == from)) return GEMM_ERR_UNSUPPORTED;
    }
    for (const Span &o : others)
        if (o.from && hit(o.from, o.to)) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Whether the norm or the workspace, which a call writes, shares memory with a
// gradient or with the other.
gemm_status check_written(int64_t n, const void *const *src, const int64_t *sizes, const int *types, Span norm, Span ws) {
    auto meet = [](const Span &a, const Span &b) { return a.from && b.from && a.from < b.to && b.from < a.to; };
    if (meet(norm, ws)) return GEMM_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        const Span g = span_of(src[i], (size_t)(sizes[i] * elem_size(types[i])));
        if (meet(g, norm) || meet(g, ws)) return GEMM_ERR_UNSUPPORTED;
    }
    return GEMM_OK;
}

// The scaling of all tensors, the last table first.
template <int MOST>
gemm_status scale(int64_t n, const void *const *src, void *const *dst, const int64_t *sizes, const int *types,
                  float max_norm, const float *given, float *norm, const double *part, int parts, hipStream_t s) {
    // Results beyond the caches' size are streamed past them (fp32 1 GiB: 583 ->
    // 556 us for norm and scaling).
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += sizes[i] * elem_size(types[i]);
    const bool stream_out = bytes >= (int64_t)256 << 20;
    int64_t starts[kMostGrads / tg::kGradTable + 1];
    int tables = 0;
    tg::GradTable<MOST> t;
    for (int64_t at = 0; at < n;) {
        const int64_t next = fill(t, at, n, src, dst, sizes, types);
        if (t.count == 0) break;
        starts[tables++] = at;
        at = next;
    }
    if (tables == 0) {                                 // (no elements: the norm alone)
        t.count = 0;
        t.first[0] = 0;
        hipLaunchKernelGGL(tg::grad_scale_kernel<MOST>, dim3(1), dim3(256), 0, s, t, part, parts, given, max_norm, norm,
                           false);
        return launched(hipGetLastError());
    }
    for (int k = tables - 1; k >= 0; --k) {
        if (k < tables - 1) fill(t, starts[k], n, src, dst, sizes, types);
        hipLaunchKernelGGL(tg::grad_scale_kernel<MOST>, dim3(groups(t)), dim3(256), 0, s, t, part, parts, given,
                           max_norm, k == 0 ? norm : nullptr, stream_out);
        const gemm_status st = launched(hipGetLastError());
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

// f(integral_constant<int, MOST>): the table for n tensors.  A launch with the
// small one passes 0.5 KiB of arguments in place of 3.7.
template <class F>
gemm_status with_table(int64_t n, F &&f) {
    if (n <= tg::kGradFew) return f(std::integral_constant<int, tg::kGradFew>());
    return f(std::integral_constant<int, tg::kGradTable>());
}

gemm_status check_room(int64_t n, const void *ws, size_t bytes) {
    if (!ws || bytes < grad_workspace_bytes(n)) return GEMM_ERR_WORKSPACE;
    return (uintptr_t)ws % 256 != 0 ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

}  // namespace

extern "C" {

size_t grad_workspace_bytes(int64_t n) {
    if (n < 0 || n >= kMostGrads) return 0;
    return (size_t)((n + tg::kGradTable - 1) / tg::kGradTable + 1) * tg::kGradGroups * sizeof(double);
}

gemm_status grad_norm(int64_t n, const void *const *grads, const int64_t *sizes, const int *types, float *norm,
                      void *workspace, size_t workspace_bytes, hipStream_t stream) {
    gemm_status st = check_grads(n, grads, nullptr, sizes, types);
    if (st != GEMM_OK) return st;
    if (!norm) return GEMM_ERR_NULL_POINTER;
    if (misaligned(norm, 4)) return GEMM_ERR_MISALIGNED;
    if ((st = check_room(n, workspace, workspace_bytes)) != GEMM_OK) return st;
    st = check_written(n, grads, sizes, types, span_of(norm, 4), span_of(workspace, grad_workspace_bytes(n)));
    if (st != GEMM_OK) return st;
    int parts;
    st = with_table(n, [&](auto most) {
        return squares<decltype(most)::value>(n, grads, sizes, types, (double *)workspace, &parts, stream);
    });
    if (st != GEMM_OK) return st;
    hipLaunchKernelGGL(tg::grad_norm_kernel, dim3(1), dim3(256), 0, stream, (const double *)workspace, parts, norm);
    return launched(hipGetLastError());
}

gemm_status grad_clip(int64_t n, const void *const *grads, void *const *out, const int64_t *sizes, const int *types,
                      float max_norm, const float *given, float *norm, void *workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    gemm_status st = check_grads(n, grads, out, sizes, types);
    if (st != GEMM_OK) return st;
    if (!(max_norm >= 0.0f)) return GEMM_ERR_UNSUPPORTED;
    if (!given && !norm) return GEMM_ERR_NULL_POINTER;
    if (misaligned(given, 4) || misaligned(norm, 4)) return GEMM_ERR_MISALIGNED;
    const Span to = span_of(norm, 4), room = span_of(given ? nullptr : workspace, grad_workspace_bytes(n));
    if ((st = check_shared(n, grads, out, sizes, types, {span_of(given, 4), to, room})) != GEMM_OK) return st;
    if ((st = check_written(n, grads, sizes, types, to, room)) != GEMM_OK) return st;
    int parts = 0;
    if (!given) {
        if ((st = check_room(n, workspace, workspace_bytes)) != GEMM_OK) return st;
        st = with_table(n, [&](auto most) {
            return squares<decltype(most)::value>(n, grads, sizes, types, (double *)workspace, &parts, stream);
        });
        if (st != GEMM_OK) return st;
    }
    if (parts > tg::kGradGroups) {
        hipLaunchKernelGGL(tg::grad_norm_kernel, dim3(1), dim3(256), 0, stream, (const double *)workspace, parts, norm);
        if ((st = launched(hipGetLastError())) != GEMM_OK) return st;
        given = norm;
    }
    return with_table(n, [&](auto most) {
        return scale<decltype(most)::value>(n, grads, out, sizes, types, max_norm, given, norm, (const double *)workspace,
                                            parts, stream);
    });
}

}  // extern "C"
