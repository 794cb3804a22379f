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
// two products whose operands have rows on 16 bytes and whole K tiles of 128
// bytes, in one launch where that is sooner; one whose D is NULL is left out
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
// tiles of 128 x 128: the same), if results per row copied are many and the copies' rows are not too long.
inline size_t prod_copy_bytes(int64_t M, int64_t N, int D, int64_t kbytes) {
    const int64_t bn = 128 / D, t128 = ((M + 127) / 128) * ((N + bn - 1) / bn);
    if (kbytes == 0 || t128 <= 512 || (double)M * (double)N * D < 300.0 * (double)(M + D * N)) return 0;
    const int64_t pitch = tg::prod_copy_pitch(kbytes);
    return pitch < kMaxLdBytes ? (size_t)(M + D * N) * (size_t)pitch : 0;
}

// Rows of an operand that the grids of all kernels hold (512 threads for 16 rows
// of B: below 2^32 in all).
constexpr int64_t kMostRows = (int64_t)1 << 27;

inline bool type16(int t) { return t == GEMM_TYPE_BF16 || t == GEMM_TYPE_FP16; }
inline bool known_act(int a) { return a >= GEMM_ACT_SILU && a <= GEMM_ACT_RELU; }

inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}
// Bytes of a rows x cols matrix, from its first element to its last.
inline int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int es) { return ((rows - 1) * ld + cols) * es; }

// A matrix in memory; whether two of them share any of it, each taken to hold
// all between its ends (`near`), or but for those whose rows are equally far
// apart and lie next to each other, as the halves of one tensor (`meet`).
struct Area {
    const void *p;
    int64_t rows, cols, ld;
    int es;
};
inline bool near(const Area &a, const Area &b) {
    return a.rows > 0 && a.cols > 0 && b.rows > 0 && b.cols > 0 &&
           overlap(a.p, matrix_bytes(a.rows, a.cols, a.ld, a.es), b.p, matrix_bytes(b.rows, b.cols, b.ld, b.es));
}
inline bool meet(const Area &a, const Area &b) {
    if (!near(a, b)) return false;
    const int64_t pitch = a.ld * a.es;
    if (a.rows == 1 || b.rows == 1 || pitch != b.ld * b.es) return true;
    const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % pitch, at = d < 0 ? d + pitch : d;
    return at < a.cols * a.es || at + b.cols * b.es > pitch;
}
inline bool near(const Area &a, const void *ws, size_t bytes) { return near(a, {ws, 1, (int64_t)bytes, (int64_t)bytes, 1}); }

}  // namespace tg_api
