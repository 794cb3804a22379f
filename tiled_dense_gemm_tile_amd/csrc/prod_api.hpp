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

// The operands copied into `ws` with rows on 16 bytes (an odd multiple of 256
// bytes apart, off each other's memory channels) and zeros up to whole chunks;
// p takes the copies.  t: the element type.
int64_t prod_copy_pitch(int64_t kbytes);
hipError_t prod_aligned_copies(ProdArgs &p, int t, char *ws, hipStream_t s);

}  // namespace tg

namespace tg_api {

// Direct loads: rows on 16 bytes and whole 16-byte chunks.
inline bool prod_aligned(const tg::ProdArgs &p) {
    auto on16 = [](const void *q, int64_t ld, int rows) {
        return (uintptr_t)q % 16 == 0 && (ld % 16 == 0 || rows == 1);
    };
    return p.KB % 16 == 0 && on16(p.A, p.lda, p.M) && on16(p.B, p.ldb, p.N) && (!p.B1 || on16(p.B1, p.ldb1, p.N));
}

// Workspace bytes of the copies of unaligned operands (M and D * N rows of
// `kbytes`), 0 where they do not pay: in grids of 256 x 256 tiles, which only
// aligned operands have (gated 4096 x 4095 x 1001: 120 us without, 78 with; 384
// tiles of 128 x 128: the same), if results per row copied are many.
inline size_t prod_copy_bytes(int64_t M, int64_t N, int D, int64_t kbytes) {
    const int64_t bn = 128 / D, t128 = ((M + 127) / 128) * ((N + bn - 1) / bn);
    if (kbytes == 0 || t128 <= 512 || (double)M * (double)N * D < 300.0 * (double)(M + D * N)) return 0;
    return (size_t)(M + D * N) * (size_t)tg::prod_copy_pitch(kbytes);
}

inline bool type16(int t) { return t == GEMM_TYPE_BF16 || t == GEMM_TYPE_FP16; }
inline bool known_act(int a) { return a >= GEMM_ACT_SILU && a <= GEMM_ACT_RELU; }

// Bytes of a rows x cols matrix, from its first element to its last.
inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}
inline int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int es) { return ((rows - 1) * ld + cols) * es; }

}  // namespace tg_api
