// Launchers of the products of prod.hpp by element type, each instantiated in
// a translation unit of its own so that they compile in parallel, and the
// host-side checks that their entry points share.
#pragma once

#include "../../include/tilegemm_layers.h"

#include "prod.hpp"
#include "rows_api.hpp"

namespace tg {

// T: 1 bf16, 2 fp16
template <int T> hipError_t launch_glu(const ProdArgs &p, const GluEpi<T> &e, hipStream_t s);
// OT: element type of D
template <int OT> hipError_t launch_int8(const ProdArgs &p, const Int8Epi<OT> &e, hipStream_t s);
// operands with rows on 16 bytes, whole K tiles of 128 bytes
template <int T, int OT> hipError_t launch_plain(const ProdArgs &p, const PlainEpi<OT> &e, hipStream_t s);
// two of them, in one launch where that is sooner
template <int T, int OT>
hipError_t launch_plain_two(const ProdArgs &p0, const PlainEpi<T> &e0, const ProdArgs &p1, const PlainEpi<OT> &e1,
                            hipStream_t s);

}  // namespace tg

namespace tg_api {

inline bool type16(int t) { return t == GEMM_TYPE_BF16 || t == GEMM_TYPE_FP16; }
inline bool known_act(int a) { return a >= GEMM_ACT_SILU && a <= GEMM_ACT_RELU; }

// Bytes of a rows x cols matrix, from its first element to its last.
inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}
inline int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int es) { return ((rows - 1) * ld + cols) * es; }

}  // namespace tg_api
