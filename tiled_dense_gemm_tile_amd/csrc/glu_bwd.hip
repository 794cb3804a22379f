// gemm_glu_backward (include/tilegemm_layers.h): checks, the kernel that makes
// the products' operands, launches.
//
// Three of the backward pass's four products sum along rows of what they are
// given (dg^T X over tokens, dg Wg over features), so their operands would be
// read across K.  One kernel lays all of them along K in the workspace, rows
// padded to whole K tiles with zeros: dg | du next to each other as M rows (A
// of the input gradient) and transposed as 2 F' rows (A of the weight
// gradients), X and Wg | Wu transposed.  Both products then run the aligned
// kernels, whatever the caller's sizes and strides, and the activation's
// derivative is computed once.  F' is F in whole tiles of 64, M' likewise.  The
// kernel is bound by memory (8192 x 14336 x 4096: 2.25 GB in 411 to 433 us, 5.2
// to 5.5 TB/s); 64 x 64 pieces, as a transposed row's 128 bytes are then whole
// lines.
//
// dg and du are rounded to the operands' 16 bits, which is what the matrix
// instructions take: relative errors of the gradients grow from 0.0017, their own
// rounding, to 0.0023 (bf16; fp16 0.00021 to 0.00029).  Kept in two pieces of 16
// bits they would double the products' instructions, 2480 of 2900 us.
#include "prod_api.hpp"

using namespace tg_api;

namespace tg {

constexpr int kCopyTile = 64;

struct GluBwdArgs {
    const void *dH, *G, *U, *X, *Wg, *Wu;
    int64_t lddh, ldg, ldu, ldx, ldwg, ldwu;
    uint16_t *dgu, *dgut, *xt, *wt;                    // (dgu, wt NULL: no input gradient; dgut, xt NULL: no weights')
    int M, F, K, Fp, Mp, act;
    int ldf, ldm;                                      // elements of a row of dgu and wt; of dgut and xt
    int tm, tf, tk;                                    // tiles of 64 along M, F, K
};

// 64 x 64 elements in LDS, rows of 64 plus two: a column's reads by 64 lanes
// (8 rows apart, eight columns) fall on distinct banks but for pairs.
constexpr int kCopyPitch = kCopyTile + 2;

// A thread's 8 elements of a row (tile row r, elements c ..) into LDS.
__device__ __forceinline__ void tile_put(uint16_t *lds, int r, int c, const uint16_t (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) *(uint32_t *)(lds + r * kCopyPitch + c + i) = v[i] | (uint32_t)v[i + 1] << 16;
}
// 8 rows' elements of column c, from row r on, as 16 bytes.
__device__ __forceinline__ u32x4 tile_column(const uint16_t *lds, int r, int c) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = lds[(r + 2 * i) * kCopyPitch + c] | (uint32_t)lds[(r + 2 * i + 1) * kCopyPitch + c] << 16;
    return v;
}

template <int T>
__global__ void __launch_bounds__(256) glu_bwd_operands_kernel(GluBwdArgs p) {
    typedef RowVec<T> R;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2][kCopyTile * kCopyPitch];
    const int tid = threadIdx.x;
    const int r0 = tid >> 3, c = (tid & 7) * 8;        // rows r0 and r0 + 32, elements c .. c + 7
    int w = blockIdx.x;
    // dg and du of 64 rows and 64 features
    const int n_act = p.tm * p.tf;
    if (w < n_act) {
        const int m0 = w / p.tf * kCopyTile, f0 = w % p.tf * kCopyTile;
        // (all loads first; past the matrix those of its last row or first
        // features, which become zeros)
        typename R::V dh[2], g[2], u[2];
        const int f = f0 + c, fc = f < p.F ? f : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t m = m0 + r0 + 32 * h < p.M ? m0 + r0 + 32 * h : p.M - 1;
            dh[h] = R::load_raw((const uint16_t *)p.dH + m * p.lddh, fc, p.F);
            g[h] = R::load_raw((const uint16_t *)p.G + m * p.ldg, fc, p.F);
            u[h] = R::load_raw((const uint16_t *)p.U + m * p.ldu, fc, p.F);
        }
        with_act(p.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = m0 + r0 + 32 * h;
                const bool in = m < p.M && f < p.F;
                const typename R::V d = R::settle(dh[h], fc, p.F), gv = R::settle(g[h], fc, p.F),
                                    uv = R::settle(u[h], fc, p.F);
                uint16_t dg[8], du[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float value, slope;
                    act_both<decltype(a)::value>(Elem<T>::up(gv[i]), value, slope);
                    const auto x = Elem<T>::down(Elem<T>::up(d[i]) * Elem<T>::up(uv[i]) * slope);
                    const auto y = Elem<T>::down(Elem<T>::up(d[i]) * value);
                    dg[i] = in && f + i < p.F ? __builtin_bit_cast(uint16_t, x) : 0;
                    du[i] = in && f + i < p.F ? __builtin_bit_cast(uint16_t, y) : 0;
                }
                if (p.dgu && m < p.M) {
                    uint16_t *row = p.dgu + (int64_t)m * p.ldf;
                    *(u32x4 *)(row + f) = __builtin_bit_cast(u32x4, dg);
                    *(u32x4 *)(row + p.Fp + f) = __builtin_bit_cast(u32x4, du);
                }
                tile_put(lds[0], r0 + 32 * h, c, dg);
                tile_put(lds[1], r0 + 32 * h, c, du);
            }
        });
        if (!p.dgut) return;
        __syncthreads();
        // feature f's tokens m0 + 8 k ..: 512 pieces of 16 bytes each
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = r0 + 32 * h, m = c;
            *(u32x4 *)(p.dgut + (int64_t)(f0 + f) * p.ldm + m0 + m) = tile_column(lds[0], m, f);
            *(u32x4 *)(p.dgut + (int64_t)(p.Fp + f0 + f) * p.ldm + m0 + m) = tile_column(lds[1], m, f);
        }
        return;
    }
    // a transposed copy: `rows` x K elements into K rows
    w -= n_act;
    const uint16_t *src;
    uint16_t *dst;
    int64_t lds_, ldd;
    int rows;
    const int n_x = p.xt ? p.tm * p.tk : 0;
    if (w < n_x) {
        src = (const uint16_t *)p.X, lds_ = p.ldx, rows = p.M, dst = p.xt, ldd = p.ldm;
    } else {
        w -= n_x;
        const int n_w = p.tf * p.tk;
        const bool up = w >= n_w;
        if (up) w -= n_w;
        src = (const uint16_t *)(up ? p.Wu : p.Wg), lds_ = up ? p.ldwu : p.ldwg, rows = p.F;
        dst = p.wt + (up ? p.Fp : 0), ldd = p.ldf;
    }
    const int a0 = w / p.tk * kCopyTile, k0 = w % p.tk * kCopyTile;
    const int k = k0 + c, kk = k < p.K ? k : 0;
    typename R::V v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t r = a0 + r0 + 32 * h < rows ? a0 + r0 + 32 * h : rows - 1;
        v[h] = R::load_raw(src + r * lds_, kk, p.K);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        u32x4 e = __builtin_bit_cast(u32x4, R::settle(v[h], kk, p.K));
        if (a0 + r0 + 32 * h >= rows) e = u32x4{0u, 0u, 0u, 0u};    // (columns past K are not stored)
#pragma unroll
        for (int i = 0; i < 4; ++i) *(uint32_t *)(lds[0] + (r0 + 32 * h) * kCopyPitch + c + 2 * i) = e[i];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = r0 + 32 * h;
        if (k0 + row < p.K) *(u32x4 *)(dst + (int64_t)(k0 + row) * ldd + a0 + c) = tile_column(lds[0], c, row);
    }
}

}  // namespace tg

namespace {

int64_t padded(int64_t n) { return (n + tg::kCopyTile - 1) / tg::kCopyTile * tg::kCopyTile; }
// Elements of a row of `n`, a multiple of 64: an odd multiple of 256 bytes.  With
// the rows of a tile a multiple of 4 KiB apart their chunks meet in few memory
// channels (8192 x 14336 x 4096: input gradient's product 1625 us with rows of
// 56 KiB, 1430 with 256 bytes more).
int64_t pitch(int64_t n) { return n + (256 + 128 - n % 256) % 256; }
int64_t part(int64_t elements) { return (elements * 2 + 255) / 256 * 256; }

// The products, the input gradient and the weights', each where it is wanted.
template <int T, int OT>
gemm_status products(const tg::GluBwdArgs &a, void *dX, int64_t lddx, const tg::PlainEpi<OT> &e, hipStream_t s) {
    tg::ProdArgs x = {}, w = {};
    x.A = a.dgu;
    x.B = a.wt;
    x.lda = x.ldb = (int64_t)a.ldf * 2;
    x.M = a.M;
    x.N = a.K;
    x.KB = a.Fp * 4;
    w.A = a.dgut;
    w.B = a.xt;
    w.lda = w.ldb = (int64_t)a.ldm * 2;
    w.M = 2 * a.Fp;
    w.N = a.K;
    w.KB = a.Mp * 2;
    const tg::PlainEpi<T> ex{{nullptr, nullptr}, {dX, nullptr}, {0, 0}, {lddx, 0}, 0x7fffffff, a.M,
                             tg::emit_whole(dX, lddx, a.K, 2), false};
    return launched(tg::launch_plain_two<T, OT>(x, ex, w, e, s));
}

template <int T>
gemm_status run(const tg::GluBwdArgs &a, void *dX, int64_t lddx, const void *Cg, int64_t ldcg, const void *Cu,
                int64_t ldcu, void *dWg, int64_t lddwg, void *dWu, int64_t lddwu, bool f32, hipStream_t s) {
    const int64_t n_act = (int64_t)a.tm * a.tf, n_x = a.xt ? (int64_t)a.tm * a.tk : 0,
                  n_w = a.wt ? 2 * (int64_t)a.tf * a.tk : 0;
    const int64_t grid = n_act + n_x + n_w;
    if (grid > 0) {
        hipLaunchKernelGGL(tg::glu_bwd_operands_kernel<T>, dim3((unsigned)grid), dim3(256), 0, s, a);
        gemm_status st = launched(hipGetLastError());
        if (st != GEMM_OK) return st;
    }
    if (a.M == 0) dX = nullptr;
    if (!dX && !dWg) return GEMM_OK;
    const int gs = f32 ? 4 : 2;
    const bool vec = tg::emit_whole(dWg, lddwg, a.K, gs) && tg::emit_whole(dWu, lddwu, a.K, gs);
    if (f32)
        return products<T, 0>(a, dX, lddx, {{Cg, Cu}, {dWg, dWu}, {ldcg, ldcu}, {lddwg, lddwu}, a.Fp, a.F, vec, Cg != nullptr}, s);
    return products<T, T>(a, dX, lddx, {{Cg, Cu}, {dWg, dWu}, {ldcg, ldcu}, {lddwg, lddwu}, a.Fp, a.F, vec, Cg != nullptr}, s);
}

}  // namespace

extern "C" {

size_t gemm_glu_backward_workspace_bytes(int64_t M, int64_t F, int64_t K) {
    if (M < 0 || F <= 0 || K <= 0 || M >= (int64_t)1 << 21 || F >= (int64_t)1 << 20 || K >= kMaxDim) return 0;
    const int64_t Fp = padded(F), ldf = pitch(2 * Fp), ldm = pitch(padded(M));
    return (size_t)(part(M * ldf) + part(2 * Fp * ldm) + part(K * ldm) + part(K * ldf));
}

gemm_status gemm_glu_backward(int64_t M, int64_t F, int64_t K, const void *dH, int64_t lddh, const void *G,
                              int64_t ldg, const void *U, int64_t ldu, const void *X, int64_t ldx, const void *Wg,
                              int64_t ldwg, const void *Wu, int64_t ldwu, int type, int act, void *dX, int64_t lddx,
                              const void *Cg, int64_t ldcg, const void *Cu, int64_t ldcu, void *dWg, int64_t lddwg,
                              void *dWu, int64_t lddwu, int grad_type, void *workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    if (M < 0 || F < 0 || K < 0) return GEMM_ERR_INVALID_SIZE;
    if (M >= (int64_t)1 << 21 || F >= (int64_t)1 << 20 || K >= kMaxDim || !type16(type) || !known_act(act) ||
        (grad_type != type && grad_type != GEMM_TYPE_F32))
        return GEMM_ERR_UNSUPPORTED;
    if ((dWg != nullptr) != (dWu != nullptr) || (Cg != nullptr) != (Cu != nullptr) || (Cg && !dWg))
        return GEMM_ERR_NULL_POINTER;
    const bool dx = dX && M > 0, dw = dWg && F > 0;
    if (K == 0 || (!dx && !dw)) return GEMM_OK;
    const int gs = elem_size(grad_type);
    if (M > 0 && F > 0 && (lddh < F || ldg < F || ldu < F)) return GEMM_ERR_BAD_LD;
    if ((dx && (lddx < K || (F > 0 && (ldwg < K || ldwu < K)))) ||
        (dw && ((M > 0 && ldx < K) || lddwg < K || lddwu < K || (Cg && (ldcg < K || ldcu < K)))))
        return GEMM_ERR_BAD_LD;
    if (M > 0 && F > 0 && (!dH || !G || !U || (dx && (!Wg || !Wu)) || (dw && !X))) return GEMM_ERR_NULL_POINTER;
    for (const void *q : {dH, G, U, X, Wg, Wu, (const void *)dX})
        if (misaligned(q, 2)) return GEMM_ERR_MISALIGNED;
    for (const void *q : {Cg, Cu, (const void *)dWg, (const void *)dWu})
        if (misaligned(q, gs)) return GEMM_ERR_MISALIGNED;
    for (int64_t ld : {lddh, ldg, ldu, dw ? ldx : 0, dx ? ldwg : 0, dx ? ldwu : 0, dx ? lddx : 0})
        if (ld * 2 >= kMaxLdBytes) return GEMM_ERR_UNSUPPORTED;
    for (int64_t ld : {dw ? lddwg : 0, dw ? lddwu : 0, Cg ? ldcg : 0, Cg ? ldcu : 0})
        if (ld * gs >= kMaxLdBytes) return GEMM_ERR_UNSUPPORTED;
    // (K is a row of the weights, so below 8 MiB too)
    // (each operand that the call reads; then Cg, Cu and the results)
    const void *const no = nullptr;
    const Area in[] = {{dH, M, F, lddh, 2}, {G, M, F, ldg, 2}, {U, M, F, ldu, 2}, {dw ? X : no, M, K, ldx, 2},
                       {dx ? Wg : no, F, K, ldwg, 2}, {dx ? Wu : no, F, K, ldwu, 2},
                       {dw ? Cg : no, F, K, ldcg, gs}, {dw ? Cu : no, F, K, ldcu, gs}};
    const Area out[] = {{dx ? dX : no, M, K, lddx, 2}, {dw ? dWg : no, F, K, lddwg, gs}, {dw ? dWu : no, F, K, lddwu, gs}};
    const bool same[] = {Cg && Cg == dWg, Cu && Cu == dWu};
    if (dw && ((same[0] && ldcg != lddwg && F > 1) || (same[1] && ldcu != lddwu && F > 1))) return GEMM_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 8; ++j)
            if (j < 6 ? near(out[i], in[j]) : !(i == j - 5 && same[j - 6]) && meet(out[i], in[j])) return GEMM_ERR_UNSUPPORTED;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return GEMM_ERR_UNSUPPORTED;
    }
    if (F == 0) {                                      // (a product without a sum: zeros)
        tg::GluBwdArgs a = {};
        a.M = (int)M;
        a.K = (int)K;
        return type == GEMM_TYPE_BF16 ? run<1>(a, dX, lddx, 0, 0, 0, 0, 0, 0, 0, 0, false, stream)
                                      : run<2>(a, dX, lddx, 0, 0, 0, 0, 0, 0, 0, 0, false, stream);
    }
    if (!workspace || workspace_bytes < gemm_glu_backward_workspace_bytes(M, F, K)) return GEMM_ERR_WORKSPACE;
    if ((uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
    const size_t used = gemm_glu_backward_workspace_bytes(M, F, K);
    for (const Area &x : in)
        if (near(x, workspace, used)) return GEMM_ERR_UNSUPPORTED;
    for (const Area &x : out)
        if (near(x, workspace, used)) return GEMM_ERR_UNSUPPORTED;
    tg::GluBwdArgs a = {};
    a.M = (int)M;
    a.F = (int)F;
    a.K = (int)K;
    a.Fp = (int)padded(F);
    a.Mp = (int)padded(M);
    a.ldf = (int)pitch(2 * (int64_t)a.Fp);
    a.ldm = (int)pitch(a.Mp);
    a.act = act;
    a.tm = a.Mp / tg::kCopyTile;
    a.tf = a.Fp / tg::kCopyTile;
    a.tk = (int)(padded(K) / tg::kCopyTile);
    a.dH = dH, a.lddh = lddh;
    a.G = G, a.ldg = ldg;
    a.U = U, a.ldu = ldu;
    a.X = X, a.ldx = ldx;
    a.Wg = Wg, a.ldwg = ldwg;
    a.Wu = Wu, a.ldwu = ldwu;
    if (((int64_t)a.tm * a.tf + (int64_t)(a.tm + 2 * a.tf) * a.tk) >= (int64_t)1 << 24) return GEMM_ERR_UNSUPPORTED;
    char *ws = (char *)workspace;
    if (dx) a.dgu = (uint16_t *)ws;
    ws += part(M * a.ldf);
    if (dw) a.dgut = (uint16_t *)ws;
    ws += part(2 * (int64_t)a.Fp * a.ldm);
    if (dw) a.xt = (uint16_t *)ws;
    ws += part(K * a.ldm);
    if (dx) a.wt = (uint16_t *)ws;
    if (type == GEMM_TYPE_BF16)
        return run<1>(a, dx ? dX : nullptr, lddx, Cg, ldcg, Cu, ldcu, dw ? dWg : nullptr, lddwg, dWu, lddwu,
                      grad_type == GEMM_TYPE_F32, stream);
    return run<2>(a, dx ? dX : nullptr, lddx, Cg, ldcg, Cu, ldcu, dw ? dWg : nullptr, lddwg, dWu, lddwu,
                  grad_type == GEMM_TYPE_F32, stream);
}

}  // extern "C"
