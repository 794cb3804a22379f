// Pieces shared by the products whose results are worked on before they are
// stored: the gated block (two products, their activation), 8-bit integers
// (scales per row and column), and the gated block's gradients.
//
// Operand rows are K-contiguous and addressed in bytes: a K tile is 128 bytes
// of a row for every type, and lane l of a 16x16 MFMA takes the 16 bytes
// 16 (l / 16) .. + 15 of 64 -- 8 elements of 16 bits (16x16x32) or 16 of 8
// (16x16x64) -- so that one set of kernels serves all of them.  B is the MFMA's
// first operand and A its second: of block (i, j) lane l holds row 16 i + l %
// 16 and the four columns 16 j + 4 (l / 16) .. + 3.
//
// PAIR (the gated block): a tile's BN rows of B are BN / 2 gate and BN / 2 up
// rows, 16 of one and then 16 of the other, so that blocks j = 2 h and 2 h + 1
// hold g and u of the same outputs in the same lane.  A load instruction fills
// 8 rows, 4 j + wave the j-th of a wave: waves 0 and 1 load gate rows, 2 and 3
// up rows, always.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "pipeline.hpp"
#include "rows.hpp"

namespace tg {

constexpr int kI8 = 3;                                 // beside the codes of gemm_elem_type

struct ProdArgs {
    const void *A, *B, *B1;                            // B1: the up rows (PAIR)
    int64_t lda, ldb, ldb1;                            // bytes
    int M, N, KB;                                      // results' rows and columns; bytes of an operand row
    int tiles_m, tiles_n, group_m;
    int run;                                           // prod_w4: tiles it computes; prod_mid, QUARTERS: the first it does not
};

// Two products in one launch.
struct ProdPair {
    ProdArgs p[2];
    int split;                                         // a multiple of 8, so that workgroups keep their XCD
};

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// acc + a.b; the sums of 8-bit integers are int32, carried in the same bits.
template <int T>
__device__ __forceinline__ f32x4 prod_mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (T == kI8)
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                                              __builtin_bit_cast(i32x4, b),
                                                                              __builtin_bit_cast(i32x4, c), 0, 0, 0));
    else if constexpr (T == 2)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// 16 bytes of an operand row from byte kb on, at any element alignment; zeros
// past the row's kbytes.
template <int T> using ProdElem = typename std::conditional<T == kI8, uint8_t, uint16_t>::type;
template <int T>
__device__ __forceinline__ u32x4 load_chunk_whole(const char *at) {
    struct __attribute__((packed, aligned(sizeof(ProdElem<T>)))) U {
        u32x4 v;
    };
    return ((const U *)at)->v;
}
// Rows of 16 bytes on, in two parts: chunk_raw has no branch and no wait, so
// that several can be in flight; it loads the row's last 16 bytes where the
// chunk would pass the row's end, and chunk_settle moves them down.
template <int T>
__device__ __forceinline__ u32x4 chunk_raw(const char *row, int kb, int kbytes) {
    return load_chunk_whole<T>(row + (kb + 16 <= kbytes ? kb : kbytes - 16));
}
__device__ __forceinline__ u32x4 chunk_settle(u32x4 v, int kb, int kbytes) {
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    const int past = kb + 16 - kbytes;                 // bytes of the chunk past the row's end
    if (past <= 0) return v;
    const u64x2 u = __builtin_bit_cast(u64x2, v);
    const uint32_t bits = 8u * (uint32_t)(past < 16 ? past : 16);
    u64x2 o;
    o[0] = bits < 64 ? (u[0] >> bits) | (u[1] << (64 - bits)) : bits < 128 ? u[1] >> (bits - 64) : 0;
    o[1] = bits < 64 ? u[1] >> bits : 0;
    return __builtin_bit_cast(u32x4, o);
}
template <int T>
__device__ __forceinline__ u32x4 load_chunk(const char *row, int kb, int kbytes) {
    if (kbytes >= 16) return chunk_settle(chunk_raw<T>(row, kb, kbytes), kb, kbytes);
    typedef ProdElem<T> E;
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int at = kb; at < kbytes; at += (int)sizeof(E)) {
        const uint64_t e = *(const E *)(row + at);
        if (at - kb < 8)
            lo |= e << (8 * (at - kb));
        else
            hi |= e << (8 * (at - kb - 8));
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// ---- results ------------------------------------------------------------------

// Four accumulators as values.  AGPR: they are read out of the AGPRs here, not
// all of them at the epilogue's start.
template <bool AGPR>
__device__ __forceinline__ f32x4 acc_value(const f32x4 &a) {
    if constexpr (AGPR) {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[r]) : "a"(a[r]));
        return v;
    } else {
        return a;
    }
}

// Floats between two rows of a wave's staged block of W columns: four banks.
template <int W> constexpr int kStagePitch = W + 4;

// Store instructions of a lane for 16 staged rows of W columns.
template <int OT, int W> constexpr int kEmitStores = 16 / (64 / (W / kVE<OT>) < 16 ? 64 / (W / kVE<OT>) : 16);

// A lane's part of 16 rows of C (element type OT, as stored).
template <int OT, int W>
struct RowsOfC {
    typename RowVec<OT>::V v[kEmitStores<OT, W>];
};

// Rows row0 .. of C (ldc 0: one row for all), loaded without a branch and ahead
// of their use: past the matrix another row's or column's.  VEC as below.
template <int OT, int W, bool VEC>
__device__ __forceinline__ void fetch_rows(RowsOfC<OT, W> &c, int lane, int row0, int col0, int M, int N, const void *C,
                                           int64_t ldc) {
    typedef RowVec<OT> R;
    constexpr int LPR = W / R::VE, RPI = 64 / LPR;
    const int lr0 = lane / LPR, col = col0 + (lane % LPR) * R::VE, at = col < N ? col : 0;
#pragma unroll
    for (int q = 0; q < kEmitStores<OT, W>; ++q) {
        const int row = row0 + q * RPI + lr0;
        const typename R::S *p = (const typename R::S *)C + (int64_t)(row < M ? row : M - 1) * ldc;
        if constexpr (VEC)
            c.v[q] = R::load_whole(p, at);
        else
            c.v[q] = R::load_raw(p, at, N);
    }
}

// 16 staged rows of W fp32 values as rows row0 .. of D (element type OT), ADD:
// plus C's: whole 16-byte pieces of a row at any element alignment.  VEC: D's
// rows start on 16 bytes and hold whole pieces; the stores are then always
// issued, kEmitStores of them (past the matrix: beyond the resource), and
// stream past the caches.
template <int OT, int W, bool VEC, bool ADD>
__device__ __forceinline__ void emit_rows(const float *stage, int lane, int row0, int col0, int M, int N, void *D,
                                          int64_t ldd, const RowsOfC<OT, W> &add) {
    typedef RowVec<OT> R;
    typedef typename R::S S;
    constexpr int VE = R::VE, LPR = W / VE, RPI = 64 / LPR;
    const int lr0 = lane / LPR, c = (lane % LPR) * VE, col = col0 + c;
    static_assert(!VEC || RPI <= 16, "whole instructions");
    const __amdgpu_buffer_rsrc_t rD =
        make_rsrc((S *)D + (int64_t)row0 * ldd, VEC ? span_bytes(M - row0 < 16 ? M - row0 : 16, N, ldd, sizeof(S)) : 0u);
    if (!VEC && col >= N) return;
#pragma unroll
    for (int q = 0; q < kEmitStores<OT, W>; ++q) {
        const int lr = q * RPI + lr0, row = row0 + lr;
        if (!VEC && ((RPI > 16 && lr >= 16) || row >= M)) continue;
        float v[VE];
#pragma unroll
        for (int h = 0; h < VE; h += 4) {
            const f32x4 t = *(const f32x4 *)(stage + lr * kStagePitch<W> + c + h);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[h + r] = t[r];
        }
        if constexpr (ADD) {
            const typename R::V a = VEC ? add.v[q] : R::settle(add.v[q], col, N);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] += Elem<OT>::up(a[i]);
        }
        typename R::V o;
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = Elem<OT>::down(v[i]);
        if constexpr (VEC)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), rD,
                                                   row < M && col < N ? (uint32_t)(lr * ldd + col) * (uint32_t)sizeof(S) : kOOB,
                                                   0, kStoreStream);
        else
            R::store((S *)D + (int64_t)row * ldd, col, N, o);
    }
}

// Whether D allows that.
inline bool emit_whole(const void *D, int64_t ldd, int64_t N, int size) {
    return (uintptr_t)D % 16 == 0 && ldd * size % 16 == 0 && N * size % 16 == 0;
}

__device__ __forceinline__ void stage_fence() {
    asm volatile("" ::: "memory");
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
}

// An epilogue has scales() and prepare(), which load into `Regs` what its
// results need and the first of C's rows, before the next tile's loads are
// issued, behind which they would wait (operations are counted in order), and
// block(), which computes and stores the results.  C's rows are loaded two blocks of 16 ahead, and nothing else is loaded
// between a tile's stores: a load there waits for the stores before it (with
// C's rows loaded where they are added, int8 8192 x 14336 x 4096 took 492 us, 390
// to 414 so, and 354 to 372 without C; gradients of 4096 x 6000 x 2048 added in
// place in fp32 490 and 418 to 430).
// (32-bit rows of 128 columns: 32 registers a block)
template <int OT> constexpr int kAheadC = OT == 0 ? 1 : 2;

// one(i, c) for the blocks in turn, fetch(c, i) AHEAD of it.
template <int TM, bool ADD, int AHEAD, class C, class Fetch, class One>
__device__ __forceinline__ void emit_blocks(C (&c)[AHEAD + 1], Fetch &&fetch, One &&one) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ADD)
            if (i + AHEAD < TM) fetch(c[(i + AHEAD) % (AHEAD + 1)], i + AHEAD);
        one(i, c[i % (AHEAD + 1)]);
    }
}

// D[m][n] = C[m][n] + sa[m] * sb[n] * sum, the int32 sum rounded to fp32 once
// (exact below 2^24) and multiplied by sa * sb, C added, then rounded to OT.
template <int OT>
struct Int8Epi {
    const float *sa, *sb;
    const void *C;
    void *D;
    int64_t ldc, ldd;
    bool vec, add;                                     // emit_whole; C given
    template <int TM, int TN> static constexpr int stores() { return TM * kEmitStores<OT, TN * 16> < 63 ? TM * kEmitStores<OT, TN * 16> : 63; }

    template <int TM, int TN>
    struct Regs {
        f32x4 cs[TN];
        float rs[TM];
        RowsOfC<OT, TN * 16> c[kAheadC<OT> + 1];
    };
    template <int TM, int TN>
    __device__ __forceinline__ void scales(Regs<TM, TN> &g, int lane, int row0, int col0, int M, int N) const {
        const int fr = lane & 15, fq = lane >> 4;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = row0 + 16 * i + fr;
            g.rs[i] = sa[m < M ? m : M - 1];
        }
#pragma unroll
        for (int j = 0; j < TN; ++j)
            g.cs[j] = RowVec<0>::load_raw(sb, col0 + 16 * j + 4 * fq < N ? col0 + 16 * j + 4 * fq : 0, N);
    }
    template <int TM, int TN, bool VEC, bool ADD>
    __device__ __forceinline__ void prepare(Regs<TM, TN> &g, int lane, int row0, int col0, int M, int N) const {
        if constexpr (ADD)
#pragma unroll
            for (int i = 0; i < kAheadC<OT> && i < TM; ++i)
                fetch_rows<OT, TN * 16, VEC>(g.c[i], lane, row0 + 16 * i, col0, M, N, C, ldc);
    }
    template <int TM, int TN, bool AGPR, bool VEC, bool ADD>
    __device__ __forceinline__ void block(Regs<TM, TN> &g, const f32x4 (&acc)[TM][TN], float *stage, int lane, int row0,
                                          int col0, int M, int N) const {
        constexpr int W = TN * 16;
        const int fr = lane & 15, fq = lane >> 4;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = col0 + 16 * j + 4 * fq;
            g.cs[j] = RowVec<0>::settle(g.cs[j], n < N ? n : 0, N);
        }
        emit_blocks<TM, ADD, kAheadC<OT>>(
            g.c,
            [&](RowsOfC<OT, W> &c, int i) __attribute__((always_inline)) {
                fetch_rows<OT, W, VEC>(c, lane, row0 + 16 * i, col0, M, N, C, ldc);
            },
            [&](int i, const RowsOfC<OT, W> &c) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const i32x4 s = __builtin_bit_cast(i32x4, acc_value<AGPR>(acc[i][j]));
                    f32x4 v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = (float)s[r] * (g.rs[i] * g.cs[j][r]);
                    *(f32x4 *)(stage + fr * kStagePitch<W> + 16 * j + 4 * fq) = v;
                }
                stage_fence();
                emit_rows<OT, W, VEC, ADD>(stage, lane, row0 + 16 * i, col0, M, N, D, ldd, c);
                stage_fence();
            });
    }
    // (result m, n of a sum's bits)
    __device__ __forceinline__ void one(int m, int n, int32_t sum) const {
        typedef typename Elem<OT>::S S;
        float v = (float)sum * (sa[m] * sb[n]);
        if (C) v += Elem<OT>::up(((const S *)C)[(int64_t)m * ldc + n]);
        ((S *)D)[(int64_t)m * ldd + n] = Elem<OT>::down(v);
    }
};

// Activations; act(g) and act'(g), from the logistic function p and the normal
// distribution's.  exp is v_exp_f32 of g log2(e): off by |g| 2^-24, relative,
// far below the 16-bit results' half step.  Where exp overflows p is 0.
enum { kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3 };

__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// 2 sqrt(2 / pi) (g + 0.044715 g^3), |g| up to 64 (beyond, p is 0 or 1 anyway,
// and the cube would overflow)
__device__ __forceinline__ float tanh_inner(float g, float &slope) {
    const float c = fminf(fmaxf(g, -64.0f), 64.0f), c2 = c * c;
    slope = 1.5957691216057308f + 0.21406452f * c2;    // 2 sqrt(2 / pi) (1 + 3 * 0.044715 g^2)
    return c * (1.5957691216057308f + 0.071354814f * c2);
}

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    float d;
    if constexpr (ACT == kSilu) return g * logistic(g);
    if constexpr (ACT == kGelu) return g * (0.5f * erfcf(g * -0.70710678118654752f));
    if constexpr (ACT == kGeluTanh) return g * logistic(tanh_inner(g, d));
    return g < 0.0f ? 0.0f : g;                        // (a NaN stays one)
}

template <int ACT>
__device__ __forceinline__ void act_both(float g, float &value, float &slope) {
    if constexpr (ACT == kSilu) {
        const float p = logistic(g);
        value = g * p;
        slope = p * (1.0f + g * (1.0f - p));
    } else if constexpr (ACT == kGelu) {
        const float p = 0.5f * erfcf(g * -0.70710678118654752f);
        value = g * p;
        slope = p + g * 0.39894228040143268f * __expf(-0.5f * g * g);
    } else if constexpr (ACT == kGeluTanh) {
        float d;
        const float p = logistic(tanh_inner(g, d));
        value = g * p;
        slope = p + g * p * (1.0f - p) * d;
    } else {
        value = g < 0.0f ? 0.0f : g;
        slope = g > 0.0f ? 1.0f : g == g ? 0.0f : g;
    }
}

// f(integral_constant<int, ACT>) of a run-time activation.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
    case kSilu: f(std::integral_constant<int, kSilu>()); break;
    case kGelu: f(std::integral_constant<int, kGelu>()); break;
    case kGeluTanh: f(std::integral_constant<int, kGeluTanh>()); break;
    default: f(std::integral_constant<int, kRelu>()); break;
    }
}

// h = act(g) * u from the fp32 sums, rounded once; G and U (NULL: not kept)
// rounded for themselves.
template <int OT>
struct GluEpi {
    void *H, *G, *U;
    int64_t ldh, ldg, ldu;
    int act;
    bool vec;
    static constexpr bool add = false;
    template <int TM, int TN> static constexpr int stores() { return TM * kEmitStores<OT, TN * 8>; }    // (H alone)

    template <int TM, int TN> struct Regs {};
    template <int TM, int TN>
    __device__ __forceinline__ void scales(Regs<TM, TN> &, int, int, int, int, int) const {}
    template <int TM, int TN, bool VEC, bool ADD>
    __device__ __forceinline__ void prepare(Regs<TM, TN> &, int, int, int, int, int) const {}
    template <int TM, int TN, bool AGPR, bool VEC, bool ADD>
    __device__ __forceinline__ void block(Regs<TM, TN> &, const f32x4 (&acc)[TM][TN], float *stage, int lane, int row0,
                                          int col0, int M, int N) const {
        constexpr int W = TN * 8;
        const int fr = lane & 15, fq = lane >> 4;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            f32x4 g[TN / 2], u[TN / 2];
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                g[j] = acc_value<AGPR>(acc[i][2 * j]);
                u[j] = acc_value<AGPR>(acc[i][2 * j + 1]);
            }
            auto put = [&](const f32x4(&v)[TN / 2], void *D, int64_t ldd) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < TN / 2; ++j) *(f32x4 *)(stage + fr * kStagePitch<W> + 16 * j + 4 * fq) = v[j];
                stage_fence();
                emit_rows<OT, W, VEC, false>(stage, lane, row0 + 16 * i, col0, M, N, D, ldd, {});
                stage_fence();
            };
            if (G) put(g, G, ldg);
            if (U) put(u, U, ldu);
            with_act(act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < TN / 2; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) g[j][r] = act_value<decltype(a)::value>(g[j][r]) * u[j][r];
            });
            put(g, H, ldh);
        }
    }
    __device__ __forceinline__ void one(int m, int n, float g, float u) const {
        typedef typename Elem<OT>::S S;
        if (G) ((S *)G)[(int64_t)m * ldg + n] = Elem<OT>::down(g);
        if (U) ((S *)U)[(int64_t)m * ldu + n] = Elem<OT>::down(u);
        with_act(act, [&](auto a) __attribute__((always_inline)) {
            ((S *)H)[(int64_t)m * ldh + n] = Elem<OT>::down(act_value<decltype(a)::value>(g) * u);
        });
    }
};

// D = sums (+ C).  Rows from `split` on go to a second matrix, as its rows 0
// ..; each has `rows` rows (a product of two stacked operands, each padded to
// `split` rows).
template <int OT>
struct PlainEpi {
    const void *C[2];
    void *D[2];
    int64_t ldc[2], ldd[2];
    int split, rows;
    bool vec, add;
    template <int TM, int TN> static constexpr int stores() { return TM * kEmitStores<OT, TN * 16> < 63 ? TM * kEmitStores<OT, TN * 16> : 63; }

    template <int TM, int TN>
    struct Regs {
        RowsOfC<OT, TN * 16> c[kAheadC<OT> + 1];
    };
    template <int TM, int TN>
    __device__ __forceinline__ void scales(Regs<TM, TN> &, int, int, int, int, int) const {}
    // (split is a multiple of 16: 16 rows lie on one side)
    template <int W, bool VEC>
    __device__ __forceinline__ void fetch(RowsOfC<OT, W> &c, int lane, int r0, int col0, int N) const {
        const int h = r0 >= split ? 1 : 0;
        fetch_rows<OT, W, VEC>(c, lane, h ? r0 - split : r0, col0, rows, N, h ? C[1] : C[0], h ? ldc[1] : ldc[0]);
    }
    template <int TM, int TN, bool VEC, bool ADD>
    __device__ __forceinline__ void prepare(Regs<TM, TN> &g, int lane, int row0, int col0, int, int N) const {
        if constexpr (ADD)
#pragma unroll
            for (int i = 0; i < kAheadC<OT> && i < TM; ++i) fetch<TN * 16, VEC>(g.c[i], lane, row0 + 16 * i, col0, N);
    }
    template <int TM, int TN, bool AGPR, bool VEC, bool ADD>
    __device__ __forceinline__ void block(Regs<TM, TN> &g, const f32x4 (&acc)[TM][TN], float *stage, int lane, int row0,
                                          int col0, int, int N) const {
        constexpr int W = TN * 16;
        const int fr = lane & 15, fq = lane >> 4;
        emit_blocks<TM, ADD, kAheadC<OT>>(
            g.c,
            [&](RowsOfC<OT, W> &c, int i) __attribute__((always_inline)) { fetch<W, VEC>(c, lane, row0 + 16 * i, col0, N); },
            [&](int i, const RowsOfC<OT, W> &c) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    *(f32x4 *)(stage + fr * kStagePitch<W> + 16 * j + 4 * fq) = acc_value<AGPR>(acc[i][j]);
                stage_fence();
                const int r0 = row0 + 16 * i, h = r0 >= split ? 1 : 0;
                emit_rows<OT, W, VEC, ADD>(stage, lane, h ? r0 - split : r0, col0, rows, N, h ? D[1] : D[0],
                                           h ? ldd[1] : ldd[0], c);
                stage_fence();
            });
    }
};

// f(VEC, ADD), as constants, of an epilogue's `vec` and `add` (C given).
template <class Epi, class F>
__device__ __forceinline__ void with_form(const Epi &e, F &&f) {
    if (e.vec) {
        if (e.add) f(std::true_type(), std::true_type());
        else f(std::true_type(), std::false_type());
    } else {
        if (e.add) f(std::false_type(), std::true_type());
        else f(std::false_type(), std::false_type());
    }
}

}  // namespace tg
