// C ABI of gemm_wgrad_mxfp8 (include/tilegemm_ops.h): checks, the choice of
// kernel and K ranges, the copy of unaligned rows, launches.
#include "../../include/tilegemm_ops.h"
#include "api.hpp"
#include "gemm_wgrad.hpp"
#include "gemm_wgrad_w4.hpp"

#include <math.h>

using namespace tg_api;

namespace {

// How a call runs: the four-wave kernel with T = 8 or 4, or (0) the one that
// takes every call, and the K ranges of its tiles (four-wave: of the tiles
// past the first `full`).
struct WgradPlan {
    int T, splits;
    int64_t full, rest;
    size_t bytes;                                      // workspace
};

constexpr int64_t kCus = 256;

// `rows16`: A and B start their rows on 16 bytes (and SFB holds four scales).
WgradPlan plan_wgrad(int64_t M, int64_t N, int64_t K, bool rows16, bool workspace) {
    WgradPlan g = {};
    const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256), t128 = ((M + 127) / 128) * ((N + 127) / 128);
    if (rows16 && K > 0) {
        auto cut = [&](int T) {                        // T x T blocks a wave: the plan
            const int64_t tiles = T == 8 ? t256 : t128, round = T == 8 ? kCus : 2 * kCus, rest = tiles % round;
            int64_t s = rest ? round / rest : 1;
            // Ranges of 1024 on; of 256 on with 128 x 128 tiles, of which
            // one's K tile takes about as long as the writing and reading of
            // a tenth of a partial sum: the least of K tiles / s and 10 s rest
            // tiles (1024 x 1024 x 1024 14.3 us uncut, 16.4 in two, 20.8 in four;
            // 512 x 512 x 8192 21.0 in eight, 23.3 in sixteen; 16 x 1920 x
            // 1382 16.8, 11.9 in two, 9.9 in five).
            const int64_t least = T == 8 ? 1024 : 256;
            if (K / least < s) s = K / least;
            if (T == 4 && rest) {
                const int64_t best = (int64_t)(sqrt(10.0 * (double)((K + 63) / 64) / (double)rest) + 0.3);
                if (best < s) s = best;
            }
            g.T = T;
            g.full = tiles;
            g.splits = 1;
            g.rest = 0;
            if (s >= 2 && workspace) {
                g.rest = rest;
                g.full = tiles - rest;
                g.splits = effective_splits(K, (int)s, 64);
            }
            g.bytes = g.splits > 1 ? (size_t)g.splits * (size_t)g.rest * (size_t)(32 * T * 32 * T) * 4 : 0;
        };
        // 256 x 256 tiles for grids of over 144 of them (136: 88 us against 80
        // with 128 x 128; 168: 89 against 98) and where fewer, cut, leave a
        // workgroup a long sum (1536 x 1536 x 16384 77 against 89 us); else
        // four times as many of 128 x 128, up to two workgroups a CU, with half the
        // partial sums (1024 x 992 x 8200 31 against 38, 2048 x 2048 x 4096
        // 45 against 49)
        if (N >= 256 && (t256 > 144 || (t256 < kCus / 2 && K / (kCus / t256) >= 1536)))
            cut(8);
        else
            cut(4);
        return g;
    }
    int64_t s = t128 ? 2 * kCus / t128 : 1;
    if (K / 256 < s) s = K / 256;
    if (s > kMaxSplits) s = kMaxSplits;
    g.splits = s < 2 || !workspace ? 1 : effective_splits(K, (int)s, 64);
    g.bytes = splitk_bytes(M, N, g.splits);
    return g;
}

// Bytes of the copy of A that puts its rows on 16 bytes, where M keeps packed
// rows off them; 0 where the kernel that takes every call is as fast (4090 x
// 4096 x 4100: 124 us with the copy, 320 without; 2001 x 992 x 2000 33 and 38;
// 3001 x 288 x 3000 32 and 32).
size_t wgrad_copy_bytes(int64_t M, int64_t N, int64_t K) {
    if (M % 8 == 0 || N < 256 || (double)M * (double)N * (double)K < 2e9) return 0;
    return (size_t)K * (size_t)((M + 7) / 8 * 8) * 2;
}

template <bool OUT_BF16, int T>
hipError_t launch_w4(const tg::Wgrad4Args &p, const tg::F16Epi &e, const WgradPlan &g, hipStream_t s) {
    hipLaunchKernelGGL((tg::gemm_wgrad_w4_kernel<OUT_BF16, T>), dim3((unsigned)(g.full + g.rest * g.splits)), dim3(256),
                       0, s, p, e);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || g.splits == 1) return err;
    hipLaunchKernelGGL((tg::wgrad_reduce_kernel<OUT_BF16, T>), dim3((unsigned)(g.rest * T * T)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

extern "C" {

size_t gemm_wgrad_mxfp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return 0;
    // (whichever kernel the operands' alignment admits)
    const size_t a = plan_wgrad(M, N, K, true, true).bytes + wgrad_copy_bytes(M, N, K);
    const size_t b = plan_wgrad(M, N, K, false, true).bytes;
    return a > b ? a : b;
}

gemm_status gemm_wgrad_mxfp8(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
                             const void *SFB, int64_t ldsfb, const void *C, int64_t ldc, void *D, int64_t ldd,
                             int out_type, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const Common a{M, N, K, A, lda, B, ldb, C, ldc, D, ldd, out_type, 1};
    bool none = false;
    gemm_status st = validate(a, &none, M, N);
    if (st != GEMM_OK) return st;
    if (N % 32 != 0) return GEMM_ERR_UNSUPPORTED;
    if (none) return GEMM_OK;
    if (lda * 2 >= kMaxLdBytes) return GEMM_ERR_UNSUPPORTED;
    if (ldsfb < N / 32) return GEMM_ERR_BAD_LD;
    if (K > 0 && !SFB) return GEMM_ERR_NULL_POINTER;
    if (misaligned(A, 2) || (uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
    // (the four-wave kernel loads four scales at once: SFB holds as many)
    const bool b16 = (((uintptr_t)B | (uintptr_t)ldb) & 15) == 0 && (K - 1) * ldsfb + N / 32 >= 4;
    bool rows16 = b16 && (((uintptr_t)A | (uintptr_t)(lda * 2)) & 15) == 0;
    if (const size_t copy = rows16 || !b16 ? 0 : wgrad_copy_bytes(M, N, K)) {
        // (behind the partial sums, which are a multiple of 16 KiB)
        const size_t at = plan_wgrad(M, N, K, true, true).bytes;
        if (workspace && workspace_bytes >= at + copy) {
            const int64_t ldo = (M + 7) / 8 * 8;
            void *out = (char *)workspace + at;
            hipLaunchKernelGGL(tg::wgrad_align_kernel,
                               dim3((unsigned)((M + 2047) / 2048), (unsigned)(K < 4096 ? K : 4096)), dim3(256), 0,
                               stream, A, lda, out, ldo, (int)K, (int)M);
            st = launched(hipGetLastError());
            if (st != GEMM_OK) return st;
            A = out;
            lda = ldo;
            rows16 = true;
        }
    }
    WgradPlan g = plan_wgrad(M, N, K, rows16, true);
    if (g.splits > 1 &&
        (!workspace || workspace_bytes < g.bytes || (!g.T && splitk_ldw(N) * 4 >= kMaxLdBytes)))
        g = plan_wgrad(M, N, K, rows16, false);
    const bool bf16 = out_type == GEMM_OUT_BF16;
    const int64_t kt = (K + 63) / 64, k_split = (kt + g.splits - 1) / g.splits * 64;
    if (g.T) {
        const int bt = 32 * g.T;
        tg::Wgrad4Args p;
        p.A = A;
        p.B = B;
        p.SF = (const uint8_t *)SFB;
        p.C = C;
        p.D = D;
        p.lda = lda;
        p.ldb = ldb;
        p.ldsf = ldsfb;
        p.ldc = ldc;
        p.ldd = ldd;
        p.M = (int)M;
        p.N = (int)N;
        p.K = (int)K;
        p.group_m = 4;
        p.tiles_m = (int)((M + bt - 1) / bt);
        p.tiles_n = (int)((N + bt - 1) / bt);
        const int64_t grid = g.full + g.rest * g.splits;
        if (grid >= kMaxDim) return GEMM_ERR_UNSUPPORTED;
        p.full = (int)g.full;
        p.splits = g.splits;
        p.k_split = (int)k_split;
        p.ws = (float *)workspace;
        const uintptr_t vb = bf16 ? 8 : 16;
        tg::F16Epi e;
        e.vec_d = ((uintptr_t)D % vb) == 0 && ldd % 4 == 0;
        e.vec_c = C && ((uintptr_t)C % vb) == 0 && ldc % 4 == 0;
        if (g.T == 8)
            return launched(bf16 ? launch_w4<true, 8>(p, e, g, stream) : launch_w4<false, 8>(p, e, g, stream));
        return launched(bf16 ? launch_w4<true, 4>(p, e, g, stream) : launch_w4<false, 4>(p, e, g, stream));
    }
    tg::WgradArgs p;
    p.A = A;
    p.B = B;
    p.SF = (const uint8_t *)SFB;
    p.C = C;
    p.D = D;
    p.lda = lda;
    p.ldb = ldb;
    p.ldsf = ldsfb;
    p.ldc = ldc;
    p.ldd = ldd;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.group_m = 8;
    p.tiles_m = (int)((M + 127) / 128);
    p.tiles_n = (int)((N + 127) / 128);
    p.ws = g.splits > 1 ? (float *)workspace : nullptr;
    p.ldw = splitk_ldw(N);
    p.k_split = (int)k_split;
    const int64_t grid = (int64_t)p.tiles_m * p.tiles_n * g.splits;
    if (grid >= kMaxDim) return GEMM_ERR_UNSUPPORTED;
    if (bf16)
        hipLaunchKernelGGL((tg::gemm_wgrad_any_kernel<true>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((tg::gemm_wgrad_any_kernel<false>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    st = launched(hipGetLastError());
    return st != GEMM_OK || g.splits == 1 ? st : reduce_splits(a, workspace, g.splits, stream);
}

}  // extern "C"
