// C ABI and kernels of gemv_mxfp4 (include/tilegemm_ops.h): a few 16-bit rows
// times 4-bit weights with group scales.
//
// Bound by the reading of W (half a byte per weight; 2 M flops per weight).
// The products run on 16x16x32 MFMAs with X as the row operand (its M rows
// padded to 16) and 16 weight rows, converted to 16 bits with their scale by
// one instruction per two, as the column operand; every product is exact
// (weights beyond fp16's range go to bf16, and fp16 X in two bf16 parts), the
// sums fp32.  Waves that share a block of weight rows along K join their sums
// through LDS in wave order; K ranges of several workgroups go through a
// workspace and are added in range order.
//
// One row of 131072 x 4096 47.8 us (5.6 TB/s of W), of 14336 x 4096 8.5 us, of
// which an empty launch is 1.6; four rows of 131072 x 8192 100 us (5.7 TB/s);
// 16 rows of 4096 x 14336 12.3 us and 2 for the ranges' sums.
#include "api.hpp"
#include "pipeline.hpp"
#include "rows.hpp"
#include "../../include/tilegemm_ops.h"

using namespace tg_api;

namespace tg {

struct GemvArgs {
    const void *X;
    const uint8_t *W, *SF;
    const void *C;
    void *D;
    int64_t ldx, ldw_bytes, ldsf, ldc, ldd;
    int M, N, K;
    int kshift;                                        // scale index of element k: k >> kshift
    int tiles_n;                                       // blocks of 16 weight rows
    bool out_bf16;
    // staged kernel: 2^kwlog waves share one block's K; LDS bytes between
    // rows of X; K per range, and where the ranges' sums go (null: one range):
    // range s to the M x ldws matrix at ws + s * M * ldws
    int kwlog, x_pitch, k_split;
    float *ws;
    int64_t ldws;
};

constexpr int kGemvWaves = 8;

struct __attribute__((packed, aligned(1))) Bytes16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(1))) Bytes8 {
    u32x2 v;
};
struct __attribute__((packed, aligned(1))) Bytes2 {
    uint16_t v;
};
struct __attribute__((packed, aligned(1))) Bytes4 {
    uint32_t v;
};
struct __attribute__((packed, aligned(2))) Halves8 {
    u32x4 v;
};

// 8 weights (one word of codes) with their scale as bf16 / fp16.
template <bool FP16>
__device__ __forceinline__ u32x4 fp4_up(uint32_t w, float scale) {
    u32x4 o;
    if constexpr (FP16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
    } else {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    }
    return o;
}

template <bool FP16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// fp16 x = hi + lo exactly, both bf16: hi holds its upper 8 significant bits,
// the remainder at most 3 (and bf16's exponents reach below fp16's).
__device__ __forceinline__ void split_f16(u32x4 x, u32x4 &hi, u32x4 &lo) {
    const f16x8 v = __builtin_bit_cast(f16x8, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = (float)v[2 * i], b = (float)v[2 * i + 1];
        hi[i] = pack_bf16x2(a, b);
        const float ra = a - __builtin_bit_cast(float, hi[i] << 16);
        const float rb = b - __builtin_bit_cast(float, hi[i] & 0xffff0000u);
        // (an infinity or NaN stays in hi alone)
        lo[i] = pack_bf16x2(__builtin_isfinite(a) ? ra : 0.0f, __builtin_isfinite(b) ? rb : 0.0f);
    }
}

// A finished sum, with C to D, or one of a K range to the workspace.
__device__ __forceinline__ void gemv_put(const GemvArgs &p, int split, int m, int n, float v) {
    if (m >= p.M || n >= p.N) return;
    if (p.ws) {
        p.ws[((int64_t)split * p.M + m) * p.ldws + n] = v;
    } else if (p.out_bf16) {
        if (p.C) v += (float)((const __bf16 *)p.C)[(int64_t)m * p.ldc + n];
        ((__bf16 *)p.D)[(int64_t)m * p.ldd + n] = (__bf16)v;
    } else {
        if (p.C) v += ((const float *)p.C)[(int64_t)m * p.ldc + n];
        ((float *)p.D)[(int64_t)m * p.ldd + n] = v;
    }
}

// The sums of each 2^kwlog neighbouring waves (one block of 16 weight rows; the
// next: the next block) joined in wave order and put.
// red[wave][4 a + r][lane]: lane l, register r holds row 16 a + 4 (l / 16) + r
// and column l % 16.
template <int MB>
__device__ __forceinline__ void gemv_join(float (&red)[kGemvWaves][MB * 4][64], const GemvArgs &p, int kwlog,
                                          int split, int m0, int n0) {
    // (through an empty asm: a persistent caller's addresses would otherwise be
    // kept in registers through its main loop)
    int first = threadIdx.x;
    asm volatile("" : "+v"(first));
    for (int i = first; i < (MB * 256 * kGemvWaves) >> kwlog; i += kGemvWaves * 64) {
        const int l = i & 63, q = (i >> 6) % (MB * 4), rw = (i >> 6) / (MB * 4), r = q & 3, a = q >> 2;
        const int m = m0 + 16 * a + 4 * (l >> 4) + r, n = n0 + 16 * rw + (l & 15);
        // (reads in asm, each waited for in its own statement: a plain LDS read
        // would also wait for the weights on their way into LDS)
        uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const float *)&red[rw << kwlog][q][l];
        float v = 0.0f;
        if (kwlog == 3) {
            float s[8];
            asm volatile(
                "ds_read_b32 %0, %8\n\tds_read_b32 %1, %8 offset:%c9\n\tds_read_b32 %2, %8 offset:%c10\n\t"
                "ds_read_b32 %3, %8 offset:%c11\n\tds_read_b32 %4, %8 offset:%c12\n\t"
                "ds_read_b32 %5, %8 offset:%c13\n\tds_read_b32 %6, %8 offset:%c14\n\t"
                "ds_read_b32 %7, %8 offset:%c15\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3]), "=&v"(s[4]), "=&v"(s[5]), "=&v"(s[6]),
                  "=&v"(s[7])
                : "v"(at), "n"(MB * 1024 * 1), "n"(MB * 1024 * 2), "n"(MB * 1024 * 3), "n"(MB * 1024 * 4),
                  "n"(MB * 1024 * 5), "n"(MB * 1024 * 6), "n"(MB * 1024 * 7)
                : "memory");
#pragma unroll
            for (int w = 0; w < 8; ++w) v += s[w];
        } else {
            for (int w = 0; w < 1 << kwlog; ++w, at += MB * 1024) {
                float s;
                asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(s) : "v"(at) : "memory");
                v += s;
            }
        }
        gemv_put(p, split, m, n, v);
    }
}

// One MFMA of 32 K: 8 weights (a word of codes) of each lane against its x.
template <bool FP16, int MB>
__device__ __forceinline__ void gemv_step(const u32x4 (&xf)[MB], uint32_t w, float scale, bool direct,
                                          f32x4 (&acc)[MB]) {
    if (!FP16 || direct) {
        const u32x4 wf = fp4_up<FP16>(w, scale);
#pragma unroll
        for (int a = 0; a < MB; ++a) acc[a] = mfma16<FP16>(xf[a], wf, acc[a]);
    } else {
        const u32x4 wf = fp4_up<false>(w, scale);
        // (weights past bf16's range meet hi alone: x that bf16 holds has lo = 0,
        // and 0 * infinity would be a NaN beside hi's infinity)
        u32x4 wl = wf;
        if (__any(scale >= 0x1p126f)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if ((wl[i] & 0x7f80u) == 0x7f80u) wl[i] &= 0xffff0000u;
                if ((wl[i] & 0x7f800000u) == 0x7f800000u) wl[i] &= 0xffffu;
            }
        }
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            u32x4 hi, lo;
            split_f16(xf[a], hi, lo);
            acc[a] = mfma16<false>(hi, wf, acc[a]);
            acc[a] = mfma16<false>(lo, wl, acc[a]);
        }
    }
}

// fp16 holds a scaled weight exactly when its scale is 2^-23 (subnormals
// included) .. 2^13; whether the lowest N codes of c are 104 .. 135, 2^-23 ..
// 2^8: 24 added to each byte (the top bits apart, so that none carries) leaves
// exactly those with the bits 100 on top.
template <int N>
__device__ __forceinline__ bool fp16_scales(uint32_t c) {
    const uint32_t v = ((c & 0x7f7f7f7fu) + 0x18181818u) ^ (c & 0x80808080u);
    constexpr uint32_t bytes = N == 4 ? 0xffffffffu : (1u << (8 * N)) - 1u;
    return (v & (0xe0e0e0e0u & bytes)) == (0x80808080u & bytes);
}

// W and X rows 16-byte aligned.  What bounds the product besides HBM is the
// count of vector-memory instructions (a 1 KiB load holds the address unit
// for about 31 cycles, whatever its lanes ask for), so X is read once per
// workgroup: a workgroup keeps its K range [k_lo, k_hi) of X in LDS and walks
// blocks of 16 weight rows (one workgroup per CU, or two).  K ranges that do not
// cover K (blockIdx.y; X too large for LDS, or too few rows for the CUs) leave
// fp32 partial sums in the workspace for a second kernel to add in order.
//
// Its eight waves share the range in steps of 256 K: KW waves take the steps
// of one block in turn, 8 / KW blocks at once.  A step's weights (16 rows of
// 128 bytes) go straight to one of the wave's own R LDS slots in whole rows,
// eight lanes a row, and are read back a word per lane in the MFMA's own
// order, in which 32 K have one scale.  Chunk c of row r sits at chunk c ^
// (r / 2 % 8): the 16 rows of a read fall on all 64 banks; rows of X are 16
// bytes longer than a multiple of 512 for the same reason.  R - 1 steps are
// requested ahead of the one being multiplied, across blocks.  Two things
// shorten that: once a turn of the ring the compiler waits for all but the
// newest one or two steps, and with C a block's end waits for C's elements and
// so for every step requested before them (131072 x 8192 for four rows, fp32 C
// and D: 100.6 us against 95.7 without C, of which 0.4 are C's bytes; all
// elements requested before the first is used made the compiler wait in calls
// without C too, 120.7).
//
// SC: groups of 32 with K % 256 == 0 (0) or not (1), of 64 (2), of 128 (3) or
// wider (4): a step's eight, eight, four, two codes or one of a row.
//
// R slots: 4; 3 where two workgroups then share a CU's LDS (X of 16 KiB at
// most: one row of 131072 x 4096 47.8 us against 55.8, of 14336 x 4096 8.5
// against 9.1, of 4096 x 4096 4.9 against 5.1), and with two blocks of 16 rows
// of X (MB; with two slots 20 rows of 28672 x 8192 42.7 against 38.4).
constexpr bool pair(int MB, int R) { return MB == 1 && R == 3; }   // two workgroups per CU
// LDS bytes a workgroup has for X beside its slots and its waves' sums.
constexpr int x_bytes(int MB, int R) {
    return (pair(MB, R) ? 80 : 160) * 1024 - kGemvWaves * 2048 * R - 2 * MB * kGemvWaves * 1024;
}

template <bool FP16, int MB, int SC, int R>
__global__ void __launch_bounds__(kGemvWaves * 64, pair(MB, R) ? 4 : 2) gemv_mxfp4_staged_kernel(GemvArgs p) {
    __shared__ __attribute__((aligned(2048))) char ring[kGemvWaves][R][2048];
    __shared__ float red[2][kGemvWaves][MB * 4][64];
    extern __shared__ __attribute__((aligned(16))) char xs[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lc = lane & 15, lg = lane >> 4;
    const int KW = 1 << p.kwlog, RW = kGemvWaves >> p.kwlog;
    const int kw = wave & (KW - 1), rw = wave >> p.kwlog;
    const int groups = (p.tiles_n + RW - 1) / RW;      // groups of RW blocks
    const int m0 = blockIdx.z * 16 * MB, rows = p.M - m0 < 16 * MB ? p.M - m0 : 16 * MB;
    const int k_lo = blockIdx.y * p.k_split, k_hi = p.K - k_lo < p.k_split ? p.K : k_lo + p.k_split;

    // ---- X's range into LDS: an instruction moves 512 elements of a row
    {
        const __amdgpu_buffer_rsrc_t r = make_rsrc((const uint16_t *)p.X + (int64_t)m0 * p.ldx + k_lo,
                                                   span_bytes(rows, k_hi - k_lo, p.ldx, 2));
        const int per_row = (k_hi - k_lo + 511) / 512;
        for (int m = 0; m < rows; ++m)
            for (int c = wave; c < per_row; c += kGemvWaves) {
                const int k = c * 512 + lane * 8;      // (whole vectors: K % 32 == 0)
                dma_load<16>(r, xs + m * p.x_pitch + c * 1024,
                             k < k_hi - k_lo ? (uint32_t)(m * p.ldx * 2) + k * 2 : kOOB);
            }
    }

    // ---- the step being requested: its group and first K (the wave's rows
    // are n0 + 16 rows of the group's)
    int rg = blockIdx.x, rk = k_lo + kw * 256;
    const uint8_t *wb, *sb;
    uint32_t wspan, so;
    auto enter = [&]() __attribute__((always_inline)) {
        const int n0 = (rg * RW + rw) * 16;
        const bool in = rg < groups && n0 < p.N;
        wb = p.W + (in ? (int64_t)n0 * p.ldw_bytes : 0);
        sb = p.SF + (in ? (int64_t)n0 * p.ldsf : 0);
        wspan = in ? span_bytes(p.N - n0, p.K / 2, p.ldw_bytes, 1) : 0u;
        const int last = in ? p.N - 1 - n0 : 0;
        so = (uint32_t)((lc < last ? lc : last) * p.ldsf);   // (rows past N: never stored)
    };
    // eight rows an instruction: lane L writes chunk L % 8 of row 8 i + L / 8
    // (rows past N lie past the resource, and so does a step past the range)
    uint32_t wo[2];
    const int wrow = lane >> 3;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wo[i] = (uint32_t)((8 * i + wrow) * p.ldw_bytes) + (((lane & 7) ^ (((8 * i + wrow) >> 1) & 7)) << 4);
    auto request_w = [&](int s) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(wb, rk < k_hi ? wspan : 0u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t o = wo[i] + (uint32_t)(rk / 2);
            if (SC != 0 && rk / 2 + (((lane & 7) ^ (((8 * i + wrow) >> 1) & 7)) << 4) >= p.K / 2) o = kOOB;
            dma_load<16>(r, ring[wave][s] + i * 1024, o);
        }
    };
    // The scales of the step in slot S, as loaded (one load, of codes inside the
    // row): they are looked at later.
    uint32_t sc[R][2];
    auto request_scales = [&](uint32_t (&c)[2]) __attribute__((always_inline)) {
        const uint8_t *sf = sb + so;
        c[1] = 0;
        if constexpr (SC <= 1) {
            const int n = p.K / 32, i = rk / 32;
            const u32x2 v = ((const Bytes8 *)(sf + (i < n - 8 ? i : n - 8)))->v;
            c[0] = v[0];
            c[1] = v[1];
        } else if constexpr (SC == 2) {
            const int n = (p.K + 63) / 64, i = rk / 64;
            c[0] = ((const Bytes4 *)(sf + (i < n - 4 ? i : n - 4)))->v;
        } else if constexpr (SC == 3) {
            const int n = (p.K + 127) / 128, i = rk / 128;
            c[0] = ((const Bytes2 *)(sf + (i < n - 2 ? i : n - 2)))->v;
        } else {
            const int last = (p.K - 1) >> p.kshift, i = rk >> p.kshift;
            c[0] = sf[i < last ? i : last];
        }
    };
    // The step at k's codes, from its load (of the row's last codes, where the
    // step's own would end past them: those before the step's drop out, and
    // blocks past K, whose weights are zeros, get 2^0): the code of K block j
    // is byte j / each.
    constexpr int each = SC <= 1 ? 1 : SC == 2 ? 2 : SC == 3 ? 4 : 8, ncodes = 8 / each;
    auto codes = [&](uint32_t (&c)[2], int k) __attribute__((always_inline)) {
        if constexpr (SC >= 1 && SC <= 3) {
            const int past = k / (32 * each) - ((p.K + 32 * each - 1) / (32 * each) - ncodes);
            if (past > 0) {
                const uint64_t v = ((uint64_t)c[1] << 32) | c[0];
                const uint64_t w = (v >> (8 * past)) | (0x7f7f7f7f7f7f7f7full << (8 * (ncodes - past)));
                c[0] = (uint32_t)w;
                c[1] = (uint32_t)(w >> 32);
            }
        }
    };

    // LDS addresses: this lane's word of chunk 0 of a slot (chunk c at ^ 16 c),
    // and its eight elements of X's first 32 (rows past M: the last row again,
    // whose sums are not stored)
    typedef __attribute__((address_space(3))) char lds_char;
    const uint32_t w0 = (uint32_t)(uintptr_t)(lds_char *)&ring[wave][0][0] + lc * 128 + ((lc >> 1) << 4) + 4 * lg;
    uint32_t x0[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const int m = 16 * a + lc < rows ? 16 * a + lc : rows - 1;
        x0[a] = (uint32_t)(uintptr_t)(lds_char *)xs + m * p.x_pitch + 16 * lg;
    }

    f32x4 acc[MB];
    int g = blockIdx.x, k0 = k_lo + kw * 256, b = 0;
    auto request = [&](auto slot) __attribute__((always_inline)) {
        constexpr int S = decltype(slot)::value;
        request_scales(sc[S]);
        request_w(S);
        rk += KW * 256;
        if (rk >= k_hi) {
            rk = k_lo + kw * 256;
            rg += gridDim.x;
            enter();
        }
    };
    // One step, of slot S; false after the workgroup's last.
    auto step = [&](auto slot) __attribute__((always_inline)) {
        constexpr int S = decltype(slot)::value;
        request(std::integral_constant<int, (S + R - 1) % R>());
        if (k0 == k_lo + kw * 256) {
#pragma unroll
            for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // this step's weights landed: only the R - 1 later steps' loads may run
        wait_vmcnt<(R - 1) * 3>();
        // (its scales are taken here in any case: left in flight on the way
        // around the branch, their registers would have the compiler wait for
        // every load)
        asm volatile("" : "+v"(sc[S][0]), "+v"(sc[S][1]) : : "memory");
        if (k0 < k_hi) {                               // (a wave past the range's last step: nothing)
            uint32_t c[2] = {sc[S][0], sc[S][1]};
            codes(c, k0);
            bool direct = true;
            if constexpr (FP16) {
                direct = fp16_scales<(ncodes < 4 ? ncodes : 4)>(c[0]);
                if constexpr (ncodes == 8) direct = direct && fp16_scales<4>(c[1]);
                direct = __all(direct);
            }
            // (reads in asm, waited for in their own statement: plain LDS reads
            // would also wait for the loads into the other slots; in two halves:
            // their registers)
            const uint32_t w = w0 + S * 2048;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t q[4];
                u32x4 xf[4][MB];
                const uint32_t x = (uint32_t)(k0 - k_lo) * 2 + 256 * h;
                asm volatile(
                    "ds_read_b32 %0, %8\n\tds_read_b32 %1, %9\n\tds_read_b32 %2, %10\n\tds_read_b32 %3, %11\n\t"
                    "ds_read_b128 %4, %12\n\tds_read_b128 %5, %12 offset:64\n\tds_read_b128 %6, %12 offset:128\n\t"
                    "ds_read_b128 %7, %12 offset:192\n\ts_waitcnt lgkmcnt(0)"
                    : "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3]), "=&v"(xf[0][0]), "=&v"(xf[1][0]),
                      "=&v"(xf[2][0]), "=&v"(xf[3][0])
                    : "v"(w ^ (64 * h)), "v"(w ^ (64 * h + 16)), "v"(w ^ (64 * h + 32)), "v"(w ^ (64 * h + 48)),
                      "v"(x0[0] + x)
                    : "memory");
                if constexpr (MB == 2)
                    asm volatile(
                        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:64\n\tds_read_b128 %2, %4 offset:128\n\t"
                        "ds_read_b128 %3, %4 offset:192\n\ts_waitcnt lgkmcnt(0)"
                        : "=&v"(xf[0][MB - 1]), "=&v"(xf[1][MB - 1]), "=&v"(xf[2][MB - 1]), "=&v"(xf[3][MB - 1])
                        : "v"(x0[MB - 1] + x)
                        : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * h + i, b = j / each;   // byte b % 4 of c[b / 4], as an exponent
                    const uint32_t v = b % 4 == 0   ? c[b / 4] << 23
                                       : b % 4 == 1 ? c[b / 4] << 15
                                       : b % 4 == 2 ? c[b / 4] << 7
                                                    : c[b / 4] >> 1;
                    gemv_step<FP16, MB>(xf[i], q[i], __builtin_bit_cast(float, v & 0x7f800000u), direct, acc);
                }
            }
        }
        k0 += KW * 256;
        if (k0 < k_hi) return true;
        k0 = k_lo + kw * 256;
        if (p.kwlog == 0) {                            // the wave's own block: no join
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    gemv_put(p, blockIdx.y, m0 + 16 * a + 4 * lg + r, (g * RW + rw) * 16 + lc, acc[a][r]);
        } else {
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int r = 0; r < 4; ++r) red[b][wave][a * 4 + r][lane] = acc[a][r];
            wait_lgkmcnt0();
            barrier();                                 // (the other half's readers passed the last one)
            gemv_join<MB>(red[b], p, p.kwlog, blockIdx.y, m0, g * RW * 16);
            b ^= 1;
        }
        g += gridDim.x;
        return g < groups;
    };

    enter();
    static_for<0, R - 1>([&](auto i) __attribute__((always_inline)) { request(i); });
    wait_vmcnt<(R - 1) * 3>();            // X landed
    barrier();
    if constexpr (R == 4) {
        while (step(std::integral_constant<int, 0>()) && step(std::integral_constant<int, 1>()) &&
               step(std::integral_constant<int, 2>()) && step(std::integral_constant<int, 3>())) {
        }
    } else {
        while (step(std::integral_constant<int, 0>()) && step(std::integral_constant<int, 1>()) &&
               step(std::integral_constant<int, 2>())) {
        }
    }
    wait_vmcnt<0>();                                   // (requests past the last group: nothing in flight into LDS at the end)
}

// Weight rows that start at any byte, K below a step, and calls without room
// for their ranges' sums.  A workgroup takes 16 weight rows and its waves share
// K; a lane's 16 bytes of a weight row are one whole 32-element block with one
// scale: K is permuted inside a step of 128 so that lane group g holds block
// g, and X is read with the same permutation.
template <bool FP16, int MB>
__global__ void __launch_bounds__(kGemvWaves * 64) gemv_mxfp4_kernel(GemvArgs p) {
    __shared__ float red[kGemvWaves][MB * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lc = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MB;
    const int K = p.K;
    // (rows past N: the last row again, never stored)
    const int64_t wrow = n0 + lc < p.N ? n0 + lc : p.N - 1;
    const uint8_t *w = p.W + wrow * p.ldw_bytes, *sf = p.SF + wrow * p.ldsf;
    const uint16_t *x[MB];
    bool xin[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        const int m = m0 + 16 * a + lc;
        xin[a] = m < p.M;
        x[a] = (const uint16_t *)p.X + (int64_t)(xin[a] ? m : 0) * p.ldx;
    }
    f32x4 acc[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a) acc[a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // wave w takes the K steps of 512 w, w + 8, ...: four tiles of 128, of
    // which lane group g loads block g, K permuted inside the tile
    for (int64_t k0 = (int64_t)wave * 512; k0 < K; k0 += kGemvWaves * 512) {
        u32x4 wq[4];
        uint32_t code[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t k = k0 + t * 128 + lg * 32;
            wq[t] = u32x4{0u, 0u, 0u, 0u};
            code[t] = 127u;
            if (k < K) {
                wq[t] = ((const Bytes16 *)(w + k / 2))->v;
                code[t] = sf[k >> p.kshift];
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t k = k0 + t * 128 + lg * 32;
            const bool direct = !FP16 || __all(fp16_scales<1>(code[t]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 xf[MB];
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    xf[a] = u32x4{0u, 0u, 0u, 0u};
                    if (xin[a] && k < K) xf[a] = ((const Halves8 *)(x[a] + k + 8 * j))->v;
                }
                gemv_step<FP16, MB>(xf, wq[t][j], __builtin_bit_cast(float, code[t] << 23), direct, acc);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][a * 4 + r][lane] = acc[a][r];
    __syncthreads();
    gemv_join<MB>(red, p, 3, 0, m0, n0);
}

struct GemvPlan {
    bool staged;
    int mb, ring, splits, k_split, kwlog;
    int64_t busiest;                                   // steps of the busiest wave
};

// Rows of X a pass of a call in several K ranges takes: its partial sums stay
// within 64 MiB (or 32 rows').
inline int64_t gemv_pass(int64_t M, int64_t N, int splits) {
    if (splits == 1) return M;
    int64_t rows = ((int64_t)64 << 20) / (splits * tg_api::splitk_ldw(N) * 4) / 32 * 32;
    if (rows < 32) rows = 32;
    return M < rows ? M : rows;
}

// The staged kernel with K ranges of ks.  Waves per block: what gives the
// busiest wave the fewest steps; among those, from ranges of 4096 on, the most
// waves that have four steps of a block each (together they read longer runs
// of its rows: 131072 x 8192 for four rows 100 us with eight waves, 113 with
// one), else the fewest (one wave needs no join and no barrier: 4096 x 14336
// for 16 rows, eight ranges of 1792, 12.4 us against 14.1 with two and 15.9
// with eight).  The count is of CUs, one workgroup each, also where two share a CU:
// they share its loads, and with 512 workgroups in the count the choice was
// slower in most calls it changed (one row of 8192 x 4096 6.1 against 6.8 us,
// of 12288 x 4096 7.9 against 8.5, of 20480 x 512 4.3 against 6.0; 28672 x 2048
// 9.3 against 8.8).
inline GemvPlan plan_ranges(int64_t M, int64_t N, int64_t K, int64_t ks) {
    GemvPlan g;
    g.staged = true;
    g.mb = M > 16 ? 2 : 1;
    g.k_split = (int)ks;
    g.splits = K > 0 ? (int)((K + ks - 1) / ks) : 1;
    const int64_t rows = M < 16 * g.mb ? M : 16 * g.mb, range = ks < K ? ks : K, steps = (range + 255) / 256;
    g.ring = g.mb == 2 ? 3 : rows * ((range + 511) / 512 * 1024 + 16) <= x_bytes(1, 3) ? 3 : 4;
    const int64_t tiles = (N + 15) / 16, tiles_m = (M + 16 * g.mb - 1) / (16 * g.mb);
    const int64_t per = 256 / (g.splits * tiles_m) > 1 ? 256 / (g.splits * tiles_m) : 1;
    g.busiest = 0;
    for (int l = 0; l <= 3; ++l) {
        const int64_t groups = (tiles + (8 >> l) - 1) / (8 >> l), each = (steps + (1 << l) - 1) >> l;
        const int64_t busiest = (groups + per - 1) / per * each;
        if (l == 0 || busiest < g.busiest || (busiest == g.busiest && steps >= 16 && each >= 4)) {
            g.busiest = busiest;
            g.kwlog = l;
        }
    }
    return g;
}

// How a call runs.  K ranges of the staged kernel: multiples of 256 (2048
// where LDS holds that much of M rows, so that all eight waves have a step of
// every block), as many as X needs; more where the blocks of rows leave half
// of the CUs idle, down to ranges of 2048; up to a quarter (and eight) more
// where the busiest wave then has fewer steps (8192 x 28672 for 16 rows 32.3 us
// against 39.0, 70000 x 8192 for two 54.8 against 58.8).
inline GemvPlan plan_gemv(int64_t M, int64_t N, int64_t K, bool aligned, bool workspace) {
    const int mb = M > 16 ? 2 : 1;
    const int64_t rows = M < 16 * mb ? M : 16 * mb;
    int64_t most = (x_bytes(mb, mb == 1 ? 4 : 3) / rows - 16) / 2 / 512 * 512;
    if (most > 2048) most = most / 2048 * 2048;
    int64_t S = K > 0 ? (K + most - 1) / most : 1;
    const int64_t tiles = (N + 15) / 16, want = 256 / (tiles < 256 ? tiles : 256);
    if (S < want && K >= 4096) S = want < K / 2048 ? want : K / 2048;
    int64_t ks = (K + S - 1) / S;
    ks = ks > 1024 ? (ks + 2047) / 2048 * 2048 : (ks + 255) / 256 * 256;
    if (ks > most) ks = most;
    GemvPlan g = plan_ranges(M, N, K, ks);
    const int64_t base = g.splits;
    for (int64_t s = base + 1; base > 1 && 4 * s <= 5 * S + 3 && s <= base + 8; ++s) {
        const GemvPlan o = plan_ranges(M, N, K, ((K + s - 1) / s + 255) / 256 * 256);
        if (o.busiest < g.busiest) g = o;
    }
    // (a step's scales are loaded together: rows hold a whole step)
    g.staged = aligned && K >= 256 && (g.splits == 1 || workspace);
    if (!g.staged) g.splits = 1;
    return g;
}

template <bool FP16, int MB, int R>
hipError_t launch_gemv(const GemvPlan &g, GemvArgs &p, hipStream_t s) {
    const dim3 threads(kGemvWaves * 64);
    const unsigned tiles_m = (unsigned)((p.M + 16 * MB - 1) / (16 * MB));
    if (!g.staged) {
        hipLaunchKernelGGL((gemv_mxfp4_kernel<FP16, MB>), dim3((unsigned)p.tiles_n, tiles_m), threads, 0, s, p);
        return hipGetLastError();
    }
    const int rows = p.M < 16 * MB ? p.M : 16 * MB;
    const int rw = kGemvWaves >> p.kwlog, groups = (p.tiles_n + rw - 1) / rw;
    const int span = p.k_split < p.K ? p.k_split : p.K;
    p.x_pitch = (span + 511) / 512 * 1024 + 16;
    int per = tg_api::cu_count(s) * (pair(MB, R) ? 2 : 1) / (int)(g.splits * tiles_m);
    if (per <= 0) per = 1;
    const dim3 grid((unsigned)(groups < per ? groups : per), (unsigned)g.splits, tiles_m);
    const size_t lds = (size_t)rows * p.x_pitch;
#define TG_GEMV(sc) hipLaunchKernelGGL((gemv_mxfp4_staged_kernel<FP16, MB, sc, R>), grid, threads, lds, s, p)
    switch (p.kshift) {
    case 5:
        if (p.K % 256 == 0)
            TG_GEMV(0);
        else
            TG_GEMV(1);
        break;
    case 6: TG_GEMV(2); break;
    case 7: TG_GEMV(3); break;
    default: TG_GEMV(4); break;
    }
#undef TG_GEMV
    return hipGetLastError();
}

template <bool FP16>
hipError_t launch_gemv_rows(const GemvPlan &g, GemvArgs &p, hipStream_t s) {
    return g.mb == 2     ? launch_gemv<FP16, 2, 3>(g, p, s)
           : g.ring == 3 ? launch_gemv<FP16, 1, 3>(g, p, s)
                         : launch_gemv<FP16, 1, 4>(g, p, s);
}

}  // namespace tg

extern "C" {

size_t gemv_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return 0;
    const int splits = tg::plan_gemv(M, N, K, true, true).splits;
    return splitk_bytes(tg::gemv_pass(M, N, splits), N, splits);
}

gemm_status gemv_mxfp4(int64_t M, int64_t N, int64_t K, int64_t kblock, const void *X, int64_t ldx, int x_type,
                       const void *W, int64_t ldw, const void *SFW, int64_t ldsfw, const void *C, int64_t ldc, void *D,
                       int64_t ldd, int out_type, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    // (X's 2-byte alignment is checked below: W's rows may start at any byte)
    const Common a{M, N, K, X, ldx, W, ldw, C, ldc, D, ldd, out_type, 1};
    bool none = false;
    gemm_status st = validate(a, &none);
    if (st != GEMM_OK || none) return st;
    if (x_type != GEMM_TYPE_BF16 && x_type != GEMM_TYPE_FP16) return GEMM_ERR_UNSUPPORTED;
    if (K % 32 != 0 || kblock <= 0 || kblock % 32 != 0 || ldw % 2 != 0) return GEMM_ERR_UNSUPPORTED;
    int kshift = 31;                                   // one scale per row: every index is 0
    if (kblock < K) {
        if ((kblock & (kblock - 1)) != 0) return GEMM_ERR_UNSUPPORTED;
        kshift = __builtin_ctzll((uint64_t)kblock);
    }
    if (ldsfw < (K + kblock - 1) / kblock) return GEMM_ERR_BAD_LD;
    if (ldsfw >= kMaxLdBytes || M > (1 << 20)) return GEMM_ERR_UNSUPPORTED;
    if (K > 0 && !SFW) return GEMM_ERR_NULL_POINTER;
    if (misaligned(X, 2) || (uintptr_t)workspace % 256 != 0) return GEMM_ERR_MISALIGNED;
    const bool aligned = (((uintptr_t)W | (uintptr_t)(ldw / 2) | (uintptr_t)X | (uintptr_t)(ldx * 2)) & 15) == 0;
    const bool room = workspace && workspace_bytes >= gemv_mxfp4_workspace_bytes(M, N, K) &&
                      splitk_ldw(N) * 4 < kMaxLdBytes;
    const tg::GemvPlan g = tg::plan_gemv(M, N, K, aligned, room);
    tg::GemvArgs p;
    p.X = X;
    p.W = (const uint8_t *)W;
    p.SF = (const uint8_t *)SFW;
    p.C = C;
    p.D = D;
    p.ldx = ldx;
    p.ldw_bytes = ldw / 2;
    p.ldsf = ldsfw;
    p.ldc = ldc;
    p.ldd = ldd;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.kshift = kshift;
    p.tiles_n = (int)((N + 15) / 16);
    p.out_bf16 = out_type == GEMM_OUT_BF16;
    p.kwlog = g.kwlog;
    p.k_split = g.k_split;
    p.x_pitch = 0;
    p.ws = g.splits > 1 ? (float *)workspace : nullptr;
    p.ldws = splitk_ldw(N);
    const int64_t pass = tg::gemv_pass(M, N, g.splits);
    for (int64_t m = 0; m < M && st == GEMM_OK; m += pass) {
        const int os = out_type == GEMM_OUT_BF16 ? 2 : 4;
        Common part = a;
        part.M = M - m < pass ? M - m : pass;
        part.A = p.X = (const char *)X + m * ldx * 2;
        if (C) part.C = p.C = (const char *)C + m * ldc * os;
        part.D = p.D = (char *)D + m * ldd * os;
        p.M = (int)part.M;
        st = launched(x_type == GEMM_TYPE_FP16 ? tg::launch_gemv_rows<true>(g, p, stream)
                                               : tg::launch_gemv_rows<false>(g, p, stream));
        if (st == GEMM_OK && g.splits > 1) st = reduce_splits(part, workspace, g.splits, stream);
    }
    return st;
}

}  // extern "C"
