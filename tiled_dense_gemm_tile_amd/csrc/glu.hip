// C ABI of gemm_glu (include/tilegemm_layers.h): checks and launch.
#include "prod_api.hpp"

using namespace tg_api;

extern "C" size_t gemm_glu_workspace_bytes(int64_t M, int64_t F, int64_t K) {
    if (M <= 0 || F <= 0 || K <= 0 || M >= kMostRows || F >= kMostRows || K * 2 >= kMaxLdBytes) return 0;
    return prod_copy_bytes(M, F, 2, K * 2);
}

extern "C" gemm_status gemm_glu(int64_t M, int64_t F, int64_t K, const void *X, int64_t ldx, const void *Wg,
                                int64_t ldwg, const void *Wu, int64_t ldwu, int type, int act, void *H, int64_t ldh,
                                void *G, int64_t ldg, void *U, int64_t ldu, void *workspace,
                                size_t workspace_bytes, hipStream_t stream) {
    if (M < 0 || F < 0 || K < 0) return GEMM_ERR_INVALID_SIZE;
    if (M >= kMostRows || F >= kMostRows || K >= kMaxDim || !type16(type) || !known_act(act)) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return GEMM_OK;
    if (ldx < K || ldwg < K || ldwu < K || ldh < F || (G && ldg < F) || (U && ldu < F)) return GEMM_ERR_BAD_LD;
    if (!H || (K > 0 && (!X || !Wg || !Wu))) return GEMM_ERR_NULL_POINTER;
    if (misaligned(X, 2) || misaligned(Wg, 2) || misaligned(Wu, 2) || misaligned(H, 2) || misaligned(G, 2) ||
        misaligned(U, 2))
        return GEMM_ERR_MISALIGNED;
    for (int64_t ld : {ldx, ldwg, ldwu, ldh, G ? ldg : 0, U ? ldu : 0})
        if (ld * 2 >= kMaxLdBytes) return GEMM_ERR_UNSUPPORTED;
    const Area at[6] = {{X, M, K, ldx, 2}, {Wg, F, K, ldwg, 2}, {Wu, F, K, ldwu, 2},
                        {H, M, F, ldh, 2}, {G, M, F, ldg, 2},   {U, M, F, ldu, 2}};
    for (int i = 3; i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (j < 3 ? near(at[i], at[j]) : meet(at[i], at[j])) return GEMM_ERR_UNSUPPORTED;
    if (workspace && (uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
    tg::ProdArgs p = {};
    p.A = X;
    p.B = Wg;
    p.B1 = Wu;
    p.lda = ldx * 2;
    p.ldb = ldwg * 2;
    p.ldb1 = ldwu * 2;
    p.M = (int)M;
    p.N = (int)F;
    p.KB = (int)(K * 2);
    const size_t need = workspace && !prod_aligned(p) ? prod_copy_bytes(M, F, 2, K * 2) : 0;
    if (need > 0 && workspace_bytes >= need) {
        for (const Area &a : at)
            if (near(a, workspace, need)) return GEMM_ERR_UNSUPPORTED;
        gemm_status st = launched(tg::prod_aligned_copies(p, type, (char *)workspace, stream));
        if (st != GEMM_OK) return st;
    }
    const bool vec = tg::emit_whole(H, ldh, F, 2) && (!G || tg::emit_whole(G, ldg, F, 2)) && (!U || tg::emit_whole(U, ldu, F, 2));
    if (type == GEMM_TYPE_BF16) return launched(tg::launch_glu<1>(p, {H, G, U, ldh, ldg, ldu, act, vec}, stream));
    return launched(tg::launch_glu<2>(p, {H, G, U, ldh, ldg, ldu, act, vec}, stream));
}
