// Host-side checks shared by the row operators (include/tilegemm_ops.h).
#pragma once

#include "../../include/tilegemm_ops.h"

#include "api.hpp"

namespace tg_api {

inline bool elem_type(int t) { return t == GEMM_TYPE_F32 || t == GEMM_TYPE_BF16 || t == GEMM_TYPE_FP16; }
inline int elem_size(int t) { return t == GEMM_TYPE_F32 ? 4 : 2; }

// Workgroups of one launch: HIP counts a grid's threads in 32 bits, so more
// rows take several launches (or a loop in the kernel).
constexpr int64_t kMaxGrid = (int64_t)1 << 20;

// rows x N sizes of a row operator; *none when there is nothing to do.
inline gemm_status check_rows(int64_t rows, int64_t N, bool *none) {
    *none = false;
    if (rows < 0 || N < 0) return GEMM_ERR_INVALID_SIZE;
    if (rows >= kMaxDim || N >= (int64_t)1 << 28) return GEMM_ERR_UNSUPPORTED;
    *none = rows == 0 || N == 0;
    return GEMM_OK;
}

}  // namespace tg_api
