// Device-side pieces of the row operators (norm, quantisation): vectors of
// 16 bytes at any element alignment, wave reductions, and the block-scaled
// output of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace tg {

// Row element types.
template <int T> struct Elem;                          // gemm_elem_type
template <> struct Elem<0> {
    typedef float S;
    static __device__ __forceinline__ float up(S v) { return v; }
    static __device__ __forceinline__ S down(float v) { return v; }
};
template <> struct Elem<1> {
    typedef __bf16 S;
    static __device__ __forceinline__ float up(S v) { return (float)v; }
    static __device__ __forceinline__ S down(float v) { return (S)v; }
};
template <> struct Elem<2> {
    typedef _Float16 S;
    static __device__ __forceinline__ float up(S v) { return (float)v; }
    static __device__ __forceinline__ S down(float v) { return (S)v; }
};

// VE = 16 bytes' worth of row elements as fp32.  The memory vector is only
// element-aligned: gfx950 serves a 16-byte access at any address, so rows
// need no padding and no scalar variant.
template <int T> constexpr int kVE = T == 0 ? 4 : 8;

template <int T>
struct RowVec {
    static constexpr int VE = kVE<T>;
    typedef typename Elem<T>::S S;
    typedef S V __attribute__((ext_vector_type(VE)));
    struct __attribute__((packed, aligned(sizeof(S)))) U {
        V v;
    };
    // As load below, the row's last vector element by element: the fewest
    // registers.
    static __device__ __forceinline__ V load_each(const void *row, int c, int n) {
        const S *p = (const S *)row + c;
        if (c + VE <= n) return ((const U *)p)->v;
        V v = {};
        for (int i = 0; i < VE; ++i)
            if (c + i < n) v[i] = p[i];
        return v;
    }
    // Elements [c, c + VE) of a row of n, 0 <= c; past the end: zeros.  The row's
    // last vector is loaded from the row's end and moved down in registers, in
    // two parts: load_raw has no branch and no wait (but in rows shorter than a
    // vector), so that several can be in flight, and settle moves.
    static __device__ __forceinline__ V load_raw(const void *row, int c, int n) {
        if (n < VE) return load_each(row, c, n);
        return ((const U *)((const S *)row + (c + VE <= n ? c : n - VE)))->v;
    }
    static __device__ __forceinline__ V settle(V v, int c, int n) {
        const int past = c + VE - n;
        if (past <= 0 || n < VE) return v;
        return down(v, past);
    }
    static __device__ __forceinline__ V load(const void *row, int c, int n) {
        return settle(load_raw(row, c, n), c, n);
    }
    // (of rows of whole vectors)
    static __device__ __forceinline__ V load_whole(const void *row, int c) { return ((const U *)((const S *)row + c))->v; }
    static __device__ __forceinline__ void store_whole(void *row, int c, V v) { ((U *)((S *)row + c))->v = v; }
    // element i + by in the place of element i, zeros on top
    static __device__ __forceinline__ V down(V v, int by) {
        typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
        const u64x2 u = __builtin_bit_cast(u64x2, v);
        const uint32_t bits = 8 * sizeof(S) * (uint32_t)by;    // >= 16
        u64x2 o;
        o[0] = bits < 64 ? (u[0] >> bits) | (u[1] << (64 - bits)) : bits < 128 ? u[1] >> (bits - 64) : 0;
        o[1] = bits < 64 ? u[1] >> bits : 0;
        return __builtin_bit_cast(V, o);
    }
    static __device__ __forceinline__ void store_each(void *row, int c, int n, V v) {
        S *p = (S *)row + c;
        if (c + VE <= n) {
            ((U *)p)->v = v;
            return;
        }
        for (int i = 0; i < VE; ++i)
            if (c + i < n) p[i] = v[i];
    }
    // (the row's end in at most three stores)
    static __device__ __forceinline__ void store(void *row, int c, int n, V v) {
        S *p = (S *)row + c;
        if (c + VE <= n) {
            ((U *)p)->v = v;
            return;
        }
        int left = n - c;
#pragma unroll
        for (int h = VE / 2; h > 0; h /= 2) {
            if (left < h) continue;
            struct __attribute__((packed, aligned(sizeof(S)))) Part {
                S s[VE];
            };
#pragma unroll
            for (int i = 0; i < h; ++i) ((Part *)p)->s[i] = v[i];
            p += h;
            left -= h;
            v = down(v, h);
        }
    }
};

// VE weights as fp32: of the row's type, or fp32 (WHOLE: rows of whole vectors).
template <int T, bool WHOLE = false>
__device__ __forceinline__ void load_weights(const void *w, bool w_f32, int c, int n, float (&out)[kVE<T>]) {
    if constexpr (T != 0) {
        if (w_f32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 v = WHOLE ? RowVec<0>::load_whole(w, c + 4 * h) : RowVec<0>::load(w, c + 4 * h, n);
#pragma unroll
                for (int i = 0; i < 4; ++i) out[4 * h + i] = v[i];
            }
            return;
        }
    }
    const auto v = WHOLE ? RowVec<T>::load_whole(w, c) : RowVec<T>::load(w, c, n);
#pragma unroll
    for (int i = 0; i < kVE<T>; ++i) out[i] = Elem<T>::up(v[i]);
}

// v of the lane at the other end of an exchange inside 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

// Sum over the wave's 64 lanes, the same in every lane: exchanges inside 16
// lanes run in the vector pipe, the last two through the LDS crossbar.
__device__ __forceinline__ float wave_sum(float v) {
    v += __builtin_bit_cast(float, dpp<kXor1>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(float, dpp<kXor2>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(float, dpp<kMirror8>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(float, dpp<kMirror16>(__builtin_bit_cast(uint32_t, v)));
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// 64-bit values of another lane: any, and one at the other end of an exchange
// inside 16 lanes.
__device__ __forceinline__ double shfl_xor64(double v, int by) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((uint32_t)u, by), hi = __shfl_xor((uint32_t)(u >> 32), by);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, ((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32) | dpp<CTRL>((uint32_t)u));
}

// As wave_sum, of 64-bit values.
__device__ __forceinline__ double wave_sum64(double v) {
    v += dpp64<kXor1>(v);
    v += dpp64<kXor2>(v);
    v += dpp64<kMirror8>(v);
    v += dpp64<kMirror16>(v);
    v += shfl_xor64(v, 16);
    v += shfl_xor64(v, 32);
    return v;
}

// Bits of |v|, or 0 for a NaN or an infinity: as unsigned numbers they order
// like the magnitudes.
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// e8m0 code of the least power of two 2^e with amax <= 448 * 2^e = 1.75 *
// 2^(e + 8): adding 0x1fffff to the bits carries into the exponent exactly
// when the significand is above 1.75, and the exponent field less 8 is then
// e + 127 (held at 0, 2^-127).
__device__ __forceinline__ uint32_t mx_code(uint32_t amax_bits) {
    const uint32_t f = (amax_bits + 0x1fffffu) >> 23;
    return f > 8u ? f - 8u : 0u;
}

// 2^(127 - code), what an element is multiplied with before its rounding
// (code <= 247: a normal number).
__device__ __forceinline__ float mx_inverse(uint32_t code) {
    return __builtin_bit_cast(float, (254u - code) << 23);
}

// VE consecutive elements of a row, their 32-element block spread over 32 /
// VE neighbouring lanes: codes and scale of the row's block-scaled form.
// (Values are at most 448 here, where the conversion neither saturates nor
// makes a NaN of its own; infinities become the NaN code.)
template <int VE, bool STREAM = false>
__device__ __forceinline__ void mx_store(const float (&y)[VE], uint8_t *q, uint8_t *sf, int c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        const uint32_t b = finite_bits(y[i]);
        m = m > b ? m : b;
    }
    auto join = [&](uint32_t o) __attribute__((always_inline)) { m = m > o ? m : o; };
    join(dpp<kXor1>(m));
    join(dpp<kXor2>(m));
    if constexpr (VE == 4) join(dpp<kMirror8>(m));
    const uint32_t code = mx_code(m);
    const float inv = mx_inverse(code);
    struct __attribute__((packed, aligned(1))) Words {
        uint32_t w[VE / 4];
    } out;
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[i] * inv, y[i + 1] * inv, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[i + 2] * inv, y[i + 3] * inv, w, true);
        out.w[i / 4] = (uint32_t)w;
    }
    if constexpr (STREAM) {
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) __builtin_nontemporal_store(out.w[i], &((Words *)(q + c))->w[i]);
    } else {
        *(Words *)(q + c) = out;
    }
    if (c % 32 == 0) sf[c / 32] = (uint8_t)code;
}

}  // namespace tg
