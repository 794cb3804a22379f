// C ABI and kernels of rmsnorm_backward (include/tilegemm_ops.h).
//
// With u = h * rstd (the normed row) and g = dy * w:
//     dx = dh + rstd * (g - u * mean(g * u))          dw = sum over rows of dy * u
// One pass over dy and h: a workgroup walks rows with a fixed set of columns
// per thread, so a row needs one reduction (mean(g * u)) and a thread's share
// of dw stays in registers over all its rows.  Each workgroup's dw goes to
// the workspace and a second kernel adds those partial sums in order: no
// atomics, the same bits on every call.  Bound by the HBM rate: 16384 x 4096
// bf16 with dh 102 us, 5.3 TB/s (97 and 5 for the two kernels); 1001 x 4100
// fp32 14 us.
#include "rows.hpp"
#include "rows_api.hpp"

using namespace tg_api;

namespace tg {

struct NormBwdArgs {
    const void *dY, *H, *W, *dH;
    const float *rstd;
    void *dX;
    float *part;                                       // gridDim.x rows of N, or null
    int64_t lddy, ldh, lddh, lddx;
    int64_t rows;
    int N;
    bool w_f32;
};

// TPR threads per row of a workgroup of NT (64: a wave, NT / 64 rows at once),
// VPT vectors of 16 bytes per thread.  The next row's vectors are loaded
// before the current one's reduction where the registers hold both.
template <int T, int TPR, int NT, int VPT>
__global__ void __launch_bounds__(NT) rmsnorm_bwd_kernel(NormBwdArgs p) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE, RPB = NT / TPR, WPR = TPR / 64;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, N = p.N;
    __shared__ float part[2][RPB][WPR];
    float w[VPT][VE], dw[VPT][VE];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * VE;
#pragma unroll
        for (int u = 0; u < VE; ++u) w[i][u] = dw[i][u] = 0.0f;
        if (c < N) load_weights<T>(p.W, p.w_f32, c, N, w[i]);
    }
    constexpr bool AHEAD = VPT <= 2;                   // (two rows of four vectors do not fit the registers)
    struct Row {
        typename RV::V dy[VPT], h[VPT], a[VPT];
        float rstd;
    };
    // (loaded ahead: settled when used; at once, but element by element, where
    // the registers are short)
    auto get = [&](const typename RV::S *row, int c) __attribute__((always_inline)) {
        return AHEAD ? RV::load_raw(row, c, N) : RV::load_each(row, c, N);
    };
    auto load = [&](int64_t row, Row &r) __attribute__((always_inline)) {
        r.rstd = 0.0f;
        if (row < p.rows) r.rstd = p.rstd[row];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * VE;
            r.dy[i] = r.h[i] = r.a[i] = typename RV::V{};
            if (row < p.rows && c < N) {
                r.dy[i] = get((const typename RV::S *)p.dY + row * p.lddy, c);
                r.h[i] = get((const typename RV::S *)p.H + row * p.ldh, c);
                if (p.dH) r.a[i] = get((const typename RV::S *)p.dH + row * p.lddh, c);
            }
        }
    };
    Row cur, next;
    if constexpr (AHEAD) load((int64_t)blockIdx.x * RPB + sub, cur);
    int slot = 0;
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < p.rows; first += (int64_t)gridDim.x * RPB, slot ^= 1) {
        const int64_t row = first + sub;
        if constexpr (AHEAD)
            load(row + (int64_t)gridDim.x * RPB, next);
        else
            load(row, cur);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * VE;
            if (AHEAD && c < N && c + VE > N) {        // the row's last vector
                cur.dy[i] = RV::settle(cur.dy[i], c, N);
                cur.h[i] = RV::settle(cur.h[i], c, N);
                cur.a[i] = RV::settle(cur.a[i], c, N);
            }
#pragma unroll
            for (int u = 0; u < VE; ++u) {
                const float d = Elem<T>::up(cur.dy[i][u]), f = Elem<T>::up(cur.h[i][u]) * cur.rstd;
                dw[i][u] = fmaf(d, f, dw[i][u]);
                m = fmaf(d * w[i][u], f, m);
            }
        }
        m = wave_sum(m);
        if constexpr (WPR > 1) {
            if ((t & 63) == 0) part[slot][sub][t >> 6] = m;
            __syncthreads();                           // (the other slot's readers passed the last one)
            m = 0.0f;
#pragma unroll
            for (int v = 0; v < WPR; ++v) m += part[slot][sub][v];
        }
        m /= (float)N;
        if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * TPR + t) * VE;
                if (c < N) {
                    typename RV::V o;
#pragma unroll
                    for (int u = 0; u < VE; ++u) {
                        const float g = Elem<T>::up(cur.dy[i][u]) * w[i][u], f = Elem<T>::up(cur.h[i][u]) * cur.rstd;
                        o[u] = Elem<T>::down(fmaf(cur.rstd, g - f * m, Elem<T>::up(cur.a[i][u])));
                    }
                    typename RV::S *dx = (typename RV::S *)p.dX + row * p.lddx;
                    if constexpr (AHEAD)
                        RV::store(dx, c, N, o);
                    else
                        RV::store_each(dx, c, N, o);
                }
            }
        }
        if constexpr (AHEAD) cur = next;
    }
    if (!p.part) return;
    // this workgroup's dw: of several rows at once, their shares added in order
    if constexpr (RPB > 1) {
        __shared__ float share[RPB][TPR * VPT * VE];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int u = 0; u < VE; ++u) share[sub][(i * TPR + t) * VE + u] = dw[i][u];
        __syncthreads();
        for (int c = threadIdx.x; c < N; c += NT) {
            float v = 0.0f;
#pragma unroll
            for (int s = 0; s < RPB; ++s) v += share[s][c];
            p.part[(int64_t)blockIdx.x * N + c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * VE;
#pragma unroll
            for (int h = 0; h < VE; h += 4)
                if (c < N)
                    RowVec<0>::store(p.part + (int64_t)blockIdx.x * N, c + h, N,
                                     f32x4{dw[i][h], dw[i][h + 1], dw[i][h + 2], dw[i][h + 3]});
        }
    }
}

// Rows too long for one workgroup's registers: dw first (its own reading of
// dy and h: dX may be dY), then dx in two passes over each row.
template <int T>
__global__ void __launch_bounds__(256) rmsnorm_bwd_dw_long_kernel(NormBwdArgs p, int groups) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VE;
    if (c >= p.N) return;
    float dw[VE] = {};
    for (int64_t row = blockIdx.y; row < p.rows; row += groups) {
        const float rstd = p.rstd[row];
        const typename RV::V dy = RV::load((const typename RV::S *)p.dY + row * p.lddy, (int)c, p.N);
        const typename RV::V h = RV::load((const typename RV::S *)p.H + row * p.ldh, (int)c, p.N);
#pragma unroll
        for (int u = 0; u < VE; ++u) dw[u] = fmaf(Elem<T>::up(dy[u]), Elem<T>::up(h[u]) * rstd, dw[u]);
    }
#pragma unroll
    for (int h = 0; h < VE; h += 4)
        RowVec<0>::store(p.part + (int64_t)blockIdx.y * p.N, (int)c + h, p.N,
                         f32x4{dw[h], dw[h + 1], dw[h + 2], dw[h + 3]});
}

template <int T>
__device__ __forceinline__ void rmsnorm_bwd_dx_long_row(const NormBwdArgs &p, int64_t row) {
    typedef RowVec<T> RV;
    constexpr int VE = RV::VE;
    const int t = threadIdx.x, N = p.N;
    const float rstd = p.rstd[row];
    const typename RV::S *dys = (const typename RV::S *)p.dY + row * p.lddy;
    const typename RV::S *hs = (const typename RV::S *)p.H + row * p.ldh;
    float m = 0.0f;
    for (int64_t c = (int64_t)t * VE; c < N; c += 1024 * VE) {
        const typename RV::V dy = RV::load(dys, (int)c, N), h = RV::load(hs, (int)c, N);
        float w[VE];
        load_weights<T>(p.W, p.w_f32, (int)c, N, w);
#pragma unroll
        for (int u = 0; u < VE; ++u) m = fmaf(Elem<T>::up(dy[u]) * w[u], Elem<T>::up(h[u]) * rstd, m);
    }
    __shared__ float part[16];
    m = wave_sum(m);
    if ((t & 63) == 0) part[t >> 6] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int v = 0; v < 16; ++v) m += part[v];
    m /= (float)N;
    for (int64_t c = (int64_t)t * VE; c < N; c += 1024 * VE) {
        const typename RV::V dy = RV::load(dys, (int)c, N), h = RV::load(hs, (int)c, N);
        typename RV::V a = {}, o;
        if (p.dH) a = RV::load((const typename RV::S *)p.dH + row * p.lddh, (int)c, N);
        float w[VE];
        load_weights<T>(p.W, p.w_f32, (int)c, N, w);
#pragma unroll
        for (int u = 0; u < VE; ++u) {
            const float g = Elem<T>::up(dy[u]) * w[u], f = Elem<T>::up(h[u]) * rstd;
            o[u] = Elem<T>::down(fmaf(rstd, g - f * m, Elem<T>::up(a[u])));
        }
        RV::store((typename RV::S *)p.dX + row * p.lddx, (int)c, N, o);
    }
}

template <int T>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_dx_long_kernel(NormBwdArgs p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        rmsnorm_bwd_dx_long_row<T>(p, row);
        __syncthreads();                               // (the row's sums in LDS)
    }
}

// dW[n] = sum over the G partial rows, in order within each of 32 lanes'
// strided shares and then over the lanes: 32 columns per workgroup, 128-byte
// runs of a partial row per load.
__global__ void __launch_bounds__(256) rmsnorm_bwd_reduce_kernel(const float *part, int G, int N, float *dW) {
    __shared__ float sums[32][33];
    const int cl = threadIdx.x & 7, r = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 32 + cl * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < N) {
        int g = r;
        for (; g + 7 * 32 < G; g += 8 * 32) {          // (eight loads in flight)
            f32x4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = RowVec<0>::load(part + (int64_t)(g + 32 * i) * N, (int)c, N);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; g < G; g += 32) s += RowVec<0>::load(part + (int64_t)g * N, (int)c, N);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[r][cl * 4 + i] = s[i];
    __syncthreads();
    const int col = threadIdx.x;
    if (col < 32 && (int64_t)blockIdx.x * 32 + col < N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sums[i][col];
        dW[(int64_t)blockIdx.x * 32 + col] = v;
    }
}

// Workgroups walking the rows: two per CU, or one where a thread has several
// vectors in flight anyway or the rows are few (fewer partial sums of dw: 1000
// x 8192 bf16 18.5 against 24.1 us, 4096 x 14336 74 against 81, 1000 x 4096
// 11.9 against 13.9; 4096 x 4096 28.6 against 26.6, 16384 x 2048 39.5 against
// 37.2).
constexpr int kBwdGroups = 512;
constexpr int kLongGroups = 64;

template <int T>
hipError_t launch_bwd(const NormBwdArgs &p, float *dW, hipStream_t s) {
    const int nvec = (int)(((int64_t)p.N + kVE<T> - 1) / kVE<T>);
    int G = 0;
    if (p.rows > 0) {
        // (rows of 16-bit elements past 16384 do not fit the registers)
#define TG_BWD(tpr, nt, vpt)                                                                                     \
    {                                                                                                            \
        const int64_t blocks = (p.rows + (nt) / (tpr) - 1) / ((nt) / (tpr));                                     \
        const int64_t most = (vpt) > 1 || blocks < 2048 ? kBwdGroups / 2 : kBwdGroups;                           \
        G = (int)(blocks < most ? blocks : most);                                                                \
        hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, tpr, nt, vpt>), dim3(G), dim3(nt), 0, s, p);                   \
    }
        if (nvec <= 64) {
            TG_BWD(64, 512, 1)
        } else if (nvec <= 128) {
            TG_BWD(128, 512, 1)
        } else if (nvec <= 256) {
            TG_BWD(256, 512, 1)
        } else if (nvec <= 512) {
            TG_BWD(512, 512, 1)
        } else if (nvec <= 1024) {
            TG_BWD(512, 512, 2)
        } else if (nvec <= 2048) {
            // (16-bit rows: 1024 threads of two vectors spill)
            if constexpr (T == 0)
                TG_BWD(1024, 1024, 2)
            else
                TG_BWD(512, 512, 4)
        } else if (T == 0 && nvec <= 4096) {
            if constexpr (T == 0) TG_BWD(1024, 1024, 4)
        } else {
            G = (int)(p.rows < kLongGroups ? p.rows : kLongGroups);
            if (p.part) {
                hipLaunchKernelGGL((rmsnorm_bwd_dw_long_kernel<T>), dim3((nvec + 255) / 256, G), dim3(256), 0, s, p, G);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            hipLaunchKernelGGL((rmsnorm_bwd_dx_long_kernel<T>), dim3((unsigned)(p.rows < 2048 ? p.rows : 2048)),
                               dim3(1024), 0, s, p);
        }
#undef TG_BWD
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dW) {
        const unsigned grid = (unsigned)(((int64_t)p.N + 31) / 32);
        hipLaunchKernelGGL(rmsnorm_bwd_reduce_kernel, dim3(grid), dim3(256), 0, s, p.part, G, p.N, dW);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace tg

extern "C" {

size_t rmsnorm_backward_workspace_bytes(int64_t rows, int64_t N) {
    bool none;
    if (check_rows(rows, N, &none) != GEMM_OK || none) return 0;
    return (size_t)(rows < tg::kBwdGroups ? rows : tg::kBwdGroups) * (size_t)N * 4;
}

gemm_status rmsnorm_backward(int64_t rows, int64_t N, const void *dY, int64_t lddy, const void *H, int64_t ldh,
                             int type, const void *W, int w_type, const float *rstd, const void *dH, int64_t lddh,
                             void *dX, int64_t lddx, float *dW, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    bool none;
    gemm_status st = check_rows(rows, N, &none);
    if (st != GEMM_OK) return st;
    if (!elem_type(type) || (w_type != type && w_type != GEMM_TYPE_F32)) return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || (none && !dW)) return GEMM_OK;
    if (misaligned(dW, 4)) return GEMM_ERR_MISALIGNED;
    tg::NormBwdArgs p = {};
    p.rows = rows;
    p.N = (int)N;
    if (rows > 0) {
        if (lddy < N || ldh < N || (dH && lddh < N) || lddx < N) return GEMM_ERR_BAD_LD;
        if (!dY || !H || !W || !rstd || !dX) return GEMM_ERR_NULL_POINTER;
        const int es = elem_size(type);
        if (misaligned(dY, es) || misaligned(H, es) || misaligned(dH, es) || misaligned(dX, es) ||
            misaligned(W, elem_size(w_type)) || misaligned(rstd, 4))
            return GEMM_ERR_MISALIGNED;
        if ((dX == dY && lddx != lddy) || (dX == dH && lddx != lddh) || dX == H) return GEMM_ERR_UNSUPPORTED;
        if (dW) {
            if (!workspace || workspace_bytes < rmsnorm_backward_workspace_bytes(rows, N)) return GEMM_ERR_WORKSPACE;
            if ((uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
        }
        p.dY = dY;
        p.H = H;
        p.W = W;
        p.dH = dH;
        p.rstd = rstd;
        p.dX = dX;
        p.part = dW ? (float *)workspace : nullptr;
        p.lddy = lddy;
        p.ldh = ldh;
        p.lddh = lddh;
        p.lddx = lddx;
        p.w_f32 = w_type == GEMM_TYPE_F32;
    }
    hipError_t e;
    switch (type) {
    case GEMM_TYPE_F32: e = tg::launch_bwd<0>(p, dW, stream); break;
    case GEMM_TYPE_BF16: e = tg::launch_bwd<1>(p, dW, stream); break;
    default: e = tg::launch_bwd<2>(p, dW, stream); break;
    }
    return launched(e);
}

}  // extern "C"
