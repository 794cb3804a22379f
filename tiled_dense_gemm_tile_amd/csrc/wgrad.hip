// C ABI of gemm_wgrad_mxfp8 (include/tilegemm_ops.h): checks, the choice of
// kernel and K ranges, launches.
#include "../../include/tilegemm_ops.h"
#include "api.hpp"
#include "gemm_wgrad.hpp"

using namespace tg_api;

namespace {

// K ranges of a call: as many as fill the GPU's 256 CUs with 128 x 128 tiles
// two deep, each of at least 1024 rows.
int wgrad_splits(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    int64_t s = tiles ? 512 / tiles : 1;
    if (K / 1024 < s) s = K / 1024;
    if (s > kMaxSplits) s = kMaxSplits;
    return s < 2 ? 1 : effective_splits(K, (int)s, 64);
}

}  // namespace

extern "C" {

size_t gemm_wgrad_mxfp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return 0;
    return splitk_bytes(M, N, wgrad_splits(M, N, K));
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
    int S = K > 0 ? wgrad_splits(M, N, K) : 1;
    if (S > 1 && (!workspace || workspace_bytes < splitk_bytes(M, N, S) || splitk_ldw(N) * 4 >= kMaxLdBytes)) S = 1;
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
    p.ws = S > 1 ? (float *)workspace : nullptr;
    p.ldw = splitk_ldw(N);
    const int64_t kt = (K + 63) / 64;
    p.k_split = (int)((kt + S - 1) / S * 64);
    const int64_t grid = (int64_t)p.tiles_m * p.tiles_n * S;
    if (grid >= kMaxDim) return GEMM_ERR_UNSUPPORTED;
    if (out_type == GEMM_OUT_BF16)
        hipLaunchKernelGGL((tg::gemm_wgrad_any_kernel<true>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((tg::gemm_wgrad_any_kernel<false>), dim3((unsigned)grid), dim3(256), 0, stream, p);
    st = launched(hipGetLastError());
    return st != GEMM_OK || S == 1 ? st : reduce_splits(a, workspace, S, stream);
}

}  // extern "C"
