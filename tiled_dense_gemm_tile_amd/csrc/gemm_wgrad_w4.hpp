// Weight gradient from block-scaled rows, four-wave kernel: output tiles of
// 256 x 256 (T = 8, one workgroup per CU) or 128 x 128 (T = 4, two), K tiles of
// 64 rows, for 16-byte rows of A and B.
//
// The MFMA schedule is the 16-bit four-wave kernel's (gemm_f16_w4.hpp: waves
// of T x T accumulator blocks of 16 x 16, K steps of 32, the second step of
// a K tile multiplied after the next tile's barrier) with both operands
// MN-contiguous: a K tile lies in LDS as 64 rows of 32 T bf16 and fragments are
// read with ds_read_b64_tr_b16.  A's tile comes by direct global -> LDS loads.
// B's tile is half as many bytes in memory and takes the registers: each
// thread loads 8 T codes of a row and its scales ahead, converts them (one
// instruction per two, with the scale) between the MFMAs of a tile's second
// half, and writes them into the slot that the tile before has left.  A
// fragment's eight K-consecutive values have eight different scales, which is
// why the conversion comes before LDS and not after it.
//
// T = 8 is bound by the MFMAs and the instructions issued between them: 14336
// x 4096 x 16384 1.40 ms, 1375 TFLOP/s (8192^3 in bf16 on the plain product's
// kernels: 1494); 4096 x 4096 x 4100 with fp32 C 128 us, of which about 30 are
// the epilogue's C and D, all tiles being of one round.  T = 4 is bound by what
// its waves wait for: small grids put one workgroup, a wave a SIMD, on most
// CUs.  1024 x 992 x 8200 28 us, 25 of them here, in which the MFMAs are busy
// for 33 % of the cycles and LDS for 35 %; 31 % of a wave's time goes to waits
// for loads, LDS and barriers, 22 % to instructions that cannot issue yet.
//
// Tiles past the last full round of workgroups (all of them, in a small grid)
// may be cut along K into `splits` ranges, whose fp32 partial tiles go to the
// workspace for a second kernel to add in order.
#pragma once

#include "common.hpp"
#include "gemm_f16_w4.hpp"
#include "gemm_wgrad.hpp"
#include "pipeline.hpp"

namespace tg {

struct Wgrad4Args {
    const void *A, *B;
    const uint8_t *SF;
    const void *C;
    void *D;
    int64_t lda, ldb, ldsf, ldc, ldd;
    int M, N, K;
    int tiles_m, tiles_n, group_m;
    int full;                                          // tiles multiplied whole: the first `full` of the walk
    int splits, k_split;                               // of the others: ranges, and K per range
    float *ws;                                         // range s of tile full + i at ws + (s * rest + i) tiles
};

// Tile `id` of the walk in groups of group_m tile rows.
__device__ __forceinline__ void walk_tile(int id, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
    const int group_size = group_m * tiles_n;
    const int group = id / group_size;
    const int first_m = group * group_m;
    const int gm = (tiles_m - first_m) < group_m ? (tiles_m - first_m) : group_m;
    const int in_group = id - group * group_size;
    tm = first_m + in_group % gm;
    tn = in_group / gm;
}

// Renumbering that gives each of the eight XCDs a run of ids.
__device__ __forceinline__ int xcd_order(int wg, int nwg) {
    const int q = nwg >> 3, r = nwg & 7, x = wg & 7;
    return x * q + (x < r ? x : r) + (wg >> 3);
}

// K tiles of `kt` rows that hold K >= 1, of any 32-bit K: K + kt - 1 would pass
// 2^31 at its end.
constexpr int k_tiles(int K, int kt) { return (K - 1) / kt + 1; }

// A half's T * T MFMAs spread B's 2 T conversion steps evenly between them; the
// step of the second half's fragment reads.
constexpr int wgrad_convert_every(int T) { return T == 8 ? 4 : 2; }
constexpr int wgrad_read_every(int T) { return T == 8 ? 3 : 1; }
// LDS operations outstanding when block row i of a tile's second half needs
// its first-half fragments (gemm_f16_w4.hpp, tr_row_wait), with the writes of
// converted B, one after every second conversion step, that the half has
// issued before its MFMA T i.
constexpr int wgrad_writes_before(int T, int q) {
    int n = 0;
    for (int s = 1; s < 2 * T; s += 2)
        if (wgrad_convert_every(T) * s + wgrad_convert_every(T) / 2 < q) ++n;
    return n;
}
constexpr int wgrad_row_wait(int T, int i) {
    const int every = wgrad_read_every(T), issued = (T * i + every - 1) / every;
    const int n = (T - 1 - i) * 2 + 2 * (issued < 2 * T ? issued : 2 * T) + wgrad_writes_before(T, T * i);
    return n > 15 ? 15 : n;
}

template <bool OUT_BF16, int T>
__global__ void __launch_bounds__(256, T == 8 ? 1 : 2) gemm_wgrad_w4_kernel(Wgrad4Args p, F16Epi e) {
    constexpr int TM = T, TN = T, BM = 32 * T, BN = 32 * T, KT = 64;
    constexpr int WTM = 16 * T, WTN = 16 * T, Q = TM * TN;
    constexpr int ROWB = BM * 2;                       // an LDS row: 32 T bf16
    constexpr int SLOT = KT * ROWB;
    // loads per thread and K tile: of A, of B, of B's scales, of C
    constexpr int LA = SLOT / 4096, NV = T / 2, NS = 1, NC = T == 8 ? 1 : 0;
    // LDS slots of A and register sets of B: a K tile of T = 4 takes less time
    // than a load, so A comes two tiles ahead and B three
    constexpr int DA = T == 8 ? 2 : 3, DB = T == 8 ? 1 : 2, UNROLL = T == 8 ? 2 : 6;
    constexpr int B_BASE = DA * SLOT;
    constexpr int RING_BYTES = (DA + 2) * SLOT;
    constexpr int EPI_BYTES = 4 * 32 * (WTN + 8) * 4;
    static_assert(RING_BYTES >= EPI_BYTES, "LDS");
    constexpr int LDS_BYTES = RING_BYTES + NC * 4096;
    static_assert(LDS_BYTES * (T == 8 ? 1 : 2) <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int rest = p.tiles_m * p.tiles_n - p.full;
    int tmi, tni, split = -1, part = 0;
    if ((int)blockIdx.x < p.full) {
        walk_tile(xcd_order(blockIdx.x, p.full), p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    } else {
        const int id = xcd_order(blockIdx.x - p.full, rest * p.splits);
        split = id / rest;
        part = id - split * rest;
        walk_tile(p.full + part, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    }
    const int m0 = tmi * BM, n0 = tni * BN;
    const int M = p.M, N = p.N;
    const int k_lo = split > 0 ? split * p.k_split : 0;
    const int K = split < 0 ? p.K : (p.K - k_lo < p.k_split ? p.K - k_lo : p.k_split);
    const int nt = k_tiles(K, KT);

    // A K tile's resource: based at its first row, ending with its last row's
    // last element (A: with the 16-byte block of it -- the range check is per
    // dword, and the block lies in the same page), moved on by 64 rows a tile.
    // All loads of a tile share it, and its few scalar instructions are spread
    // over the MFMAs (each pinned by an empty asm): built for each load, the
    // resources' ~20 scalar instructions held up the MFMAs around it (1754 us
    // at 14336 x 4096 x 16384).
    struct Panel {
        const char *base;
        uint32_t span;
        int rows;                                      // left, from base on
        __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const { return make_rsrc(base, span); }
        __device__ __forceinline__ void set_span(uint32_t ld_bytes, uint32_t row_bytes, uint32_t round) {
            const int r = rows < KT ? rows : KT;
            span = r <= 0 ? 0u : ((uint32_t)(r - 1) * ld_bytes + row_bytes + round) & ~round;
            asm volatile("" : "+s"(span));
        }
        __device__ __forceinline__ void move(int64_t step) {
            base += step;
            rows -= KT;
            asm volatile("" : "+s"(base), "+s"(rows));
        }
    };

    // ---- A: direct global -> LDS, as gemm_f16_w4t_kernel's AT operand
    Panel pa, pb;
    pa.base = (const char *)p.A + ((int64_t)k_lo * p.lda + m0) * 2;
    pa.rows = K;
    const uint32_t a_row = (uint32_t)(M - m0) * 2, a_ld = (uint32_t)(p.lda * 2);
    pa.set_span(a_ld, a_row, 15u);
    const int64_t a_step = (int64_t)KT * p.lda * 2;
    uint32_t a_off[LA];
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        constexpr int lanes = ROWB / 16;               // of one row
        const int row = 64 / lanes * (4 * j + wave) + lane / lanes;
        const int lchk = ((lane % lanes) >> 1) ^ (row & 3) ^ (((row >> 3) & 1) << 2);
        a_off[j] = (uint32_t)((row * p.lda + lchk * 16 + (lane & 1) * 8) * 2);
    }
    char *const a_lds = smem + wave * 1024;
    auto dma_a = [&](__amdgpu_buffer_rsrc_t r, int slot, int j) __attribute__((always_inline)) {
        dma_load<16>(r, a_lds + slot * SLOT + j * 4096, a_off[j]);
    };

    // ---- B: thread t holds row t / 4 of a K tile, columns 16 (t % 4) + 64 j
    // .. + 15, and their scales, the tile's in one load: T = 8: eight (the row's
    // last eight where N ends inside the tile: s_shift bits too far left); T =
    // 4: four, with what follows the row where N ends inside the tile, and the
    // matrix's last four where those would end past it.  (One load of 32 bits:
    // bytes kept across the loop are masked on arrival, and the wait for that
    // drained the loads of the tiles ahead.  Rows past K take the last row's,
    // with codes 0.)
    const int br = tid >> 2, bt = tid & 3;
    const uint32_t b_off = (uint32_t)(br * p.ldb) + bt * 16;
    const int nb = N / 32, s_at = T == 4 || n0 / 32 < nb - 8 ? n0 / 32 : nb - 8, s_shift = 8 * (n0 / 32 - s_at);
    const uint8_t *const s_end = p.SF + (int64_t)(p.K - 1) * p.ldsf + nb - 4;   // (T == 4: not before SF, wgrad.hip)
    pb.base = (const char *)p.B + (int64_t)k_lo * p.ldb + n0;
    pb.rows = K;
    const uint32_t b_row = (uint32_t)(N - n0), b_ld = (uint32_t)p.ldb;
    pb.set_span(b_ld, b_row, 0u);
    const int64_t b_step = (int64_t)KT * p.ldb;
    struct __attribute__((packed, aligned(1))) PackedScales {
        typename std::conditional<T == 8, uint64_t, uint32_t>::type v;
    };
    u32x4 vb[DB][NV];
    uint64_t vs;                                       // T == 8
    uint32_t vs4[DB], vs4_shift[DB];                   // T == 4: the scales, and the bits to this thread's first
    auto load_b = [&](__amdgpu_buffer_rsrc_t r, int set, int j) __attribute__((always_inline)) {
        vb[set][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, b_off + 64 * j, 0, 0));
    };
    const uint8_t *s_row = p.SF + (int64_t)k_lo * p.ldsf + s_at + (int64_t)(br < K ? br : K - 1) * p.ldsf;
    const int64_t s_step = (int64_t)KT * p.ldsf;
    int s_left = K - 1 - br;                           // rows from s_row's to the last
    auto load_s = [&](int set) __attribute__((always_inline)) {
        if constexpr (T == 8) {
            vs = ((const PackedScales *)s_row)->v;
        } else {
            const uint8_t *at = s_row < s_end ? s_row : s_end;
            vs4[set] = ((const PackedScales *)at)->v;
            vs4_shift[set] = 8 * ((uint32_t)(s_row - at) + (bt >> 1));
        }
    };
    auto next_s = [&]() __attribute__((always_inline)) {
        // (the row 64 further; past K: the last)
        s_left -= KT;
        s_row += s_left >= 0 ? s_step : s_left > -KT ? (int64_t)(s_left + KT) * p.ldsf : 0;
    };
    // Vector j converted, four columns a step; written as two 16-byte halves.
    // (LDS row br, 32-byte chunk bt + 4 j at ^ (br % 4) ^ 4 (br / 8 % 2), the
    // layout of A's slots)
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    uint32_t b_put[2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
        b_put[o] = lds0 + B_BASE + br * ROWB + ((bt ^ (br & 3)) + 4 * (o ^ ((br >> 3) & 1))) * 32;
    uint32_t sc[NV / 2];                               // scales of vectors 2 i and 2 i + 1 in bytes 0 and 2
    auto take_scales = [&](int set) __attribute__((always_inline)) {
        if constexpr (T == 8) {
            const uint64_t s = (vs >> s_shift) >> (8 * (bt >> 1));
            sc[0] = (uint32_t)s;
            sc[1] = (uint32_t)(s >> 32);
        } else {
            sc[0] = vs4[set] >> (vs4_shift[set] & 31);   // (32: of columns past N)
        }
    };
    u32x4 half;
    auto convert = [&](auto step, auto slot, int set) __attribute__((always_inline)) {
        constexpr int at = decltype(slot)::value * SLOT;
        constexpr int j = decltype(step)::value / 4, i = decltype(step)::value % 4;
        const float scale = __builtin_bit_cast(
            float, (j & 1) ? (sc[j / 2] & 0xff0000u) << 7 : (sc[j / 2] & 0xffu) << 23);
        half[2 * (i & 1)] =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vb[set][j][i], scale, false));
        half[2 * (i & 1) + 1] =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(vb[set][j][i], scale, true));
        if constexpr (i & 1) {
            const uint32_t put = b_put[j & 1];
            const u32x4 v = half;
            asm volatile("ds_write_b128 %0, %1 offset:%c2"
                         :
                         : "v"(put), "v"(v), "n"(at + 256 * (j / 2) + 16 * (i / 2))
                         : "memory");
        }
    };

    // ---- C's tile, which the epilogue reads: brought near the CU while the
    // matrix units are busy, a KiB a wave and K tile, into LDS that nothing
    // reads (aligned 16-byte blocks, down from its elements; past the tile, or
    // without C: no access)
    constexpr int OS = OUT_BF16 ? 2 : 4, CL = BN * OS / 16;   // blocks of a tile row
    const bool has_c = p.C && split < 0;
    const uintptr_t c_at = has_c ? (uintptr_t)p.C + ((int64_t)m0 * p.ldc + n0) * OS : 0;
    const uint32_t c_lead = (uint32_t)(c_at & 15);
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc((const void *)(c_at - c_lead),
                  has_c ? c_lead + span_bytes(M - m0 < BM ? M - m0 : BM, N - n0 < BN ? N - n0 : BN, p.ldc, OS) : 0u);
    uint32_t c_off = (uint32_t)((wave * 64 + lane) / CL * p.ldc * OS) + (lane % CL) * 16;
    const uint32_t c_step = (uint32_t)(256 / CL * p.ldc * OS);
    auto touch_c = [&]() __attribute__((always_inline)) {
        dma_load<16>(rc, smem + RING_BYTES + wave * 1024, (c_lead + c_off) & ~15u);
        c_off = c_off + c_step < 0x7fffffffu ? c_off + c_step : 0x7fffffffu;
    };

    // ---- fragments: transposing reads (gemm_f16_w4t_kernel, MN-contiguous)
    const int fr = lane & 15, fq = lane >> 4;
    auto mn_base = [&](int wb, int b) __attribute__((always_inline)) {
        const int g = (fr >> 2) ^ ((fq & 1) << 2);
        return lds0 + (8 * fq + (fr >> 2)) * ROWB + ((wb * T + b) ^ g) * 32 + (fr & 3) * 8;
    };
    uint32_t a_mn[TM], b_mn[TN];
#pragma unroll
    for (int b = 0; b < TM; ++b) a_mn[b] = mn_base(wm, b);
#pragma unroll
    for (int b = 0; b < TN; ++b) b_mn[b] = B_BASE + mn_base(wn, b);
    auto ldfrag_tr = [&](uint32_t a, auto off) __attribute__((always_inline)) {
        u32x2 lo, hi;
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%c2" : "=v"(lo) : "v"(a), "n"(decltype(off)::value));
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%c2" : "=v"(hi) : "v"(a), "n"(decltype(off)::value + 4 * ROWB));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    f32x4 acc[TM][TN];
    u32x4 fa[2][TM], fb[2][TN];                        // [K step][block]
    // of K tile I % UNROLL
    auto read_frag = [&](auto index, auto st_, int k) __attribute__((always_inline)) {
        constexpr int I = decltype(index)::value, st = decltype(st_)::value;
        constexpr std::integral_constant<int, I % DA * SLOT + st * 32 * ROWB> a_at{};
        constexpr std::integral_constant<int, I % 2 * SLOT + st * 32 * ROWB> b_at{};
        if (k == 0 || k > TN) {
            const int i = k == 0 ? 0 : k - TN;
            fa[st][i] = ldfrag_tr(a_mn[i], a_at);
        } else {
            fb[st][k - 1] = ldfrag_tr(b_mn[k - 1], b_at);
        }
    };
    auto mfma = [&](auto zero, int st, int i, int j) __attribute__((always_inline)) {
        if constexpr (decltype(zero)::value)
            mfma16_zero_asm<false>(acc[i][j], fb[st][j], fa[st][i]);
        else
            mfma16_acc_asm<false>(acc[i][j], fb[st][j], fa[st][i]);
        __builtin_amdgcn_sched_barrier(0);
    };

    // K tile t, I = t % UNROLL.  First half: step 1 of tile t - 1, with the
    // reads of tile t step 0 and the loads of A(t + DA - 1).  Second half: step
    // 0 of tile t, with the reads of step 1, the conversion of B(t + 1) (a step
    // of two instructions per four or two MFMAs, a write per two steps) and, as
    // its registers fall free, the loads of B(t + 1 + DB), which have until
    // DB tiles later's second half to land.
    auto tile = [&](auto first, auto index) __attribute__((always_inline)) {
        constexpr int I = decltype(index)::value, SET = (I + 1) % DB, RD = TM + TN;
        constexpr std::integral_constant<int, (I + 1) % 2> b_nxt{};
        constexpr std::integral_constant<int, 0> st0{};
        constexpr std::integral_constant<int, 1> st1{};
        const __amdgpu_buffer_rsrc_t ra = pa.rsrc();
        static_for<0, Q>([&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value;
            if constexpr (!decltype(first)::value) mfma(std::false_type(), 1, q / TN, q % TN);
            if constexpr (q * RD % Q == 0 && q * RD / Q < RD) read_frag(index, st0, q * RD / Q);
            if constexpr (q % (Q / LA) == (T == 8 ? 2 : 1)) dma_a(ra, (I + DA - 1) % DA, q / (Q / LA));
            if constexpr (q == (T == 8 ? 5 : 3) && !decltype(first)::value) pb.move(b_step);
            if constexpr (q == (T == 8 ? 7 : 6) && !decltype(first)::value) pb.set_span(b_ld, b_row, 0u);
            if constexpr (q == Q - 3) pa.move(a_step);
            if constexpr (q == Q - 1) pa.set_span(a_ld, a_row, 15u);
        });
        const __amdgpu_buffer_rsrc_t rb = pb.rsrc();
        static_for<0, Q>([&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q % TN == 0) __builtin_amdgcn_s_waitcnt(0xC07F | (wgrad_row_wait(T, q / TN) << 8));
            mfma(first, 0, q / TN, q % TN);
            constexpr int re = wgrad_read_every(T), ce = wgrad_convert_every(T);
            if constexpr (q % re == 0 && q / re < TM + TN) read_frag(index, st1, q / re);
            if constexpr (q == (T == 8 ? 1 : 0)) take_scales(SET);
            if constexpr (q == (T == 8 ? 5 : 2)) load_s(SET);
            if constexpr (q == (T == 8 ? 9 : 4)) next_s();
            if constexpr (q % ce == ce / 2) {
                convert(std::integral_constant<int, q / ce>(), b_nxt, SET);
                if constexpr (q / ce % 4 == 3) load_b(rb, SET, q / ce / 4);
            }
        });
        if constexpr (NC) touch_c();
        wait_vmcnt<(DA - 1) * (NV + NS + NC) + (DA - 2) * LA>();   // A(t + 1) landed; what came after it may still run
        wait_lgkmcnt0();
        barrier();
    };

    // (every K range holds a row)
    auto start_b = [&](int set) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t r = pb.rsrc();
#pragma unroll
        for (int j = 0; j < NV; ++j) load_b(r, set, j);
        load_s(set);
        next_s();
        pb.move(b_step);
        pb.set_span(b_ld, b_row, 0u);
    };
    auto start_a = [&](int slot) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t r = pa.rsrc();
#pragma unroll
        for (int j = 0; j < LA; ++j) dma_a(r, slot, j);
        pa.move(a_step);
        pa.set_span(a_ld, a_row, 15u);
    };
    start_a(0);
    start_b(0);
    if constexpr (DA == 3) start_a(1);
    if constexpr (DB == 2) start_b(1);
    take_scales(0);
    static_for<0, 2 * T>([&](auto s) __attribute__((always_inline)) {
        convert(s, std::integral_constant<int, 0>(), 0);
    });
    start_b(0);
    wait_vmcnt<(DA - 2) * LA + DB * (NV + NS)>();      // A(0) landed
    wait_lgkmcnt0();
    barrier();
    tile(std::true_type(), std::integral_constant<int, 0>());
    int t = 1;
    for (; t + UNROLL <= nt; t += UNROLL)
        static_for<0, UNROLL>([&](auto i) __attribute__((always_inline)) {
            tile(std::false_type(), std::integral_constant<int, (decltype(i)::value + 1) % UNROLL>());
        });
    // (the rest nested, each copy only behind the one before: side by side, the
    // compiler waits as if a copy could be left out)
    auto more = [&](auto self, auto i) __attribute__((always_inline)) {
        constexpr int n = decltype(i)::value;
        if constexpr (n < UNROLL) {
            if (t++ >= nt) return;
            tile(std::false_type(), i);
            self(self, std::integral_constant<int, n + 1>());
        }
    };
    more(more, std::integral_constant<int, 1>());
#pragma unroll
    for (int q = 0; q < Q; ++q) mfma(std::false_type(), 1, q / TN, q % TN);
    // (the wait states of mfma_result_fence, for either tile)
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 3" : "+a"(acc[0][0]));
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
    // (the last tiles' loads of B and its scales, which nobody multiplies: used
    // here, so that every tile issues them -- left out of a tile, as a load
    // without a use is, they would be missing from its wait's count)
#pragma unroll
    for (int d = 0; d < DB; ++d) {
#pragma unroll
        for (int j = 0; j < NV; ++j) asm volatile("" : : "v"(vb[d][j]));
        if constexpr (T == 4) asm volatile("" : : "v"(vs4[d]));
    }
    if constexpr (T == 8) asm volatile("" : : "v"(vs));
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    barrier();
    if (split < 0) {
        epilogue_lds16t<OUT_BF16, TM, TN, WTM, WTN, kStoreStream>(acc, smem, wave, lane, wm, wn, m0, n0, M, N, p.C,
                                                                  p.ldc, p.D, p.ldd, e);
    } else {
        // a whole partial tile (stays cacheable: it is read next)
        float *out = p.ws + ((int64_t)split * rest + part) * (BM * BN);
        F16Epi v;
        v.vec_c = false;
        v.vec_d = true;
        epilogue_lds16t<false, TM, TN, WTM, WTN, 0>(acc, smem, wave, lane, wm, wn, 0, 0, BM, BN, nullptr, 0, out, BN,
                                                    v);
    }
}

// D = the `splits` partial tiles of each cut tile added in order, plus C: four
// columns a thread, 1024 elements a workgroup.
template <bool OUT_BF16, int T>
__global__ void __launch_bounds__(256) wgrad_reduce_kernel(Wgrad4Args p) {
    const int rest = p.tiles_m * p.tiles_n - p.full;
    constexpr int BT = 32 * T, per_tile = BT * BT / 1024;
    const int part = blockIdx.x / per_tile, at = (blockIdx.x % per_tile) * 1024 + threadIdx.x * 4;
    int tm, tn;
    walk_tile(p.full + part, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int m = tm * BT + at / BT, n = tn * BT + at % BT;
    if (m >= p.M || n >= p.N) return;                  // (N % 32 == 0: whole vectors)
    const float *w = p.ws + (int64_t)part * (BT * BT) + at;
    const int64_t slice = (int64_t)rest * (BT * BT);
    f32x4 s = *(const f32x4 *)w;
    int k = 1;
    for (; k + 4 <= p.splits; k += 4) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *(const f32x4 *)(w + (k + i) * slice);
#pragma unroll
        for (int i = 0; i < 4; ++i) s += v[i];
    }
    for (; k < p.splits; ++k) s += *(const f32x4 *)(w + k * slice);
    wgrad_put<OUT_BF16>(s, p.C, p.ldc, p.D, p.ldd, m, n);
}

}  // namespace tg
