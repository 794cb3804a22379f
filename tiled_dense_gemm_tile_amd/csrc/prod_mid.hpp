// Products in BM x BN tiles of one workgroup, for grids too small for 256 x 256
// tiles and for operands at any alignment.
//
// KS groups of four waves (2 x 2 over the tile) take every KS-th K tile each,
// in LDS slots of their own; their sums meet in LDS at the end and are added in
// order.  Where tiles are fewer than the GPU can hold, that cuts the K loop's
// length and has KS times the loads in flight.
//
// K tiles of 128 bytes; LDS rows of 128 bytes, 16-byte chunk c of row r at
// chunk c ^ (r & 7) (free of bank conflicts for the 16-row fragment reads).
//   * Aligned operands (rows on 16 bytes, whole 16-byte chunks): S slots a
//     K tile, filled by direct global->LDS loads S - 1 tiles ahead; one barrier
//     a tile, the loads of S - 2 tiles in flight across it.
//   * ANY: the same chunks through registers (a 16-byte global load serves any
//     element alignment), PD tiles ahead of the slot they are written to; the
//     chunk at a row's end is loaded whole from there and moved down in
//     registers.  Two slots.
#pragma once

#include "prod.hpp"

namespace tg {

template <int BM, int BN, int S, int KS> constexpr int kMidLds = KS * S * (BM + BN) * 128;

// Tile (tmi, tni).
template <int T, int BM, int BN, int S, int KS, bool PAIR, bool ANY, class Epi>
__device__ __forceinline__ void prod_mid_body(const ProdArgs &p, int tmi, int tni, char *lds, const Epi &e) {
    constexpr int WTM = BM / 2, WTN = BN / 2, TM = WTM / 16, TN = WTN / 16;
    constexpr int LA = BM / 32, LB = BN / 32;          // load instructions of a wave a tile
    constexpr int SLOT_A = BM * 128, SLOT_B = BN * 128, B_BASE = S * SLOT_A;
    constexpr int GROUP = S * (SLOT_A + SLOT_B);       // LDS of a group
    constexpr int W = PAIR ? WTN / 2 : WTN;            // result columns of a wave
    constexpr int RING = KS * GROUP, STAGE = 16 * kStagePitch<W> * 4;
    constexpr int SUMS = TM * TN * 1024;               // a wave's accumulators
    static_assert(!ANY || S == 2, "ANY: two slots");
    static_assert(RING >= 4 * STAGE && RING >= (KS - 1) * 4 * SUMS + 4 * STAGE && RING <= 160 * 1024, "LDS");
    static_assert((S - 2) * (LA + LB) < 64, "vmcnt");

    const int tid = threadIdx.x, lane = tid & 63;
    const int group = KS > 1 ? __builtin_amdgcn_readfirstlane(tid >> 8) : 0;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
    char *const smem = lds + group * GROUP;
    const int wm = wave >> 1, wn = wave & 1;
    const int m0 = tmi * BM, n0 = tni * (PAIR ? BN / 2 : BN);
    const int KB = p.KB, nt = (KB + 128 * KS - 1) / (128 * KS);    // K tiles of a group: tile t is K tile KS t + group

    // Load instruction j of a wave: A rows 32 j + 8 wave + lane / 8; B the
    // same, or (PAIR) rows 16 j + 8 (wave % 2) + lane / 8 of the wave's half.
    // Lane l writes chunk l % 8 and fetches chunk (l % 8) ^ (l / 8).
    const bool up = PAIR && wave >= 2;
    const char *A = (const char *)p.A + (int64_t)m0 * p.lda;
    const int64_t ldb = up ? p.ldb1 : p.ldb;
    const char *B = (const char *)(up ? p.B1 : p.B) + (int64_t)n0 * ldb;
    const int arow = 8 * wave + (lane >> 3), brow = PAIR ? 8 * (wave & 1) + (lane >> 3) : arow;
    constexpr int BSTEP = PAIR ? 16 : 32;
    const int kc = ((lane & 7) ^ (lane >> 3)) * 16;    // byte of the tile this lane fetches

    const __amdgpu_buffer_rsrc_t rA = make_rsrc(A, span_bytes(p.M - m0, KB, p.lda, 1));
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(B, span_bytes(p.N - n0, KB, ldb, 1));
    auto dma = [&](__amdgpu_buffer_rsrc_t r, char *d, uint32_t voff, int soff) __attribute__((always_inline)) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)d, 16, voff, soff, 0, 0);
    };
    const uint32_t aoff = (uint32_t)(arow * p.lda) + kc, boff = (uint32_t)(brow * ldb) + kc;
    // (chunks past K read as zeros from an offset beyond the resource, and so
    // do all of a tile past the last, which keeps the count of loads in flight)
    auto fetch = [&](int t, int slot) __attribute__((always_inline)) {
        const int k0 = (KS * t + group) * 128;
        const bool in = k0 + kc < KB;
        const uint32_t va = in ? aoff + k0 : kOOB, vb = in ? boff + k0 : kOOB;
#pragma unroll
        for (int j = 0; j < LA; ++j)
            dma(rA, smem + slot * SLOT_A + (4 * j + wave) * 1024, va, (int)(32 * j * p.lda));
#pragma unroll
        for (int j = 0; j < LB; ++j)
            dma(rB, smem + B_BASE + slot * SLOT_B + (4 * j + wave) * 1024, vb, (int)(BSTEP * j * ldb));
    };
    // (rows past the end are read as the last one: their results are not stored)
    constexpr int PD = !ANY ? 1 : LA + LB <= 4 ? 4 : 2;
    u32x4 ra[PD][ANY ? LA : 1], rb[PD][ANY ? LB : 1];
    const char *pa[ANY ? LA : 1], *pb[ANY ? LB : 1];
    if constexpr (ANY) {
#pragma unroll
        for (int j = 0; j < LA; ++j)
            pa[j] = A + (int64_t)(arow + 32 * j < p.M - m0 ? arow + 32 * j : p.M - 1 - m0) * p.lda;
#pragma unroll
        for (int j = 0; j < LB; ++j)
            pb[j] = B + (int64_t)(brow + BSTEP * j < p.N - n0 ? brow + BSTEP * j : p.N - 1 - n0) * ldb;
    }
    auto read_any = [&](int t, int d) __attribute__((always_inline)) {
        const int kb = (KS * t + group) * 128 + kc;
#pragma unroll
        for (int j = 0; j < LA; ++j) ra[d][j] = chunk_raw<T>(pa[j], kb, KB);
#pragma unroll
        for (int j = 0; j < LB; ++j) rb[d][j] = chunk_raw<T>(pb[j], kb, KB);
    };
    auto write_any = [&](int t, int d) __attribute__((always_inline)) {
        const int slot = t & 1, k0 = (KS * t + group) * 128;
        if (KB >= 16 && k0 + 128 > KB) {
#pragma unroll
            for (int j = 0; j < LA; ++j) ra[d][j] = chunk_settle(ra[d][j], k0 + kc, KB);
#pragma unroll
            for (int j = 0; j < LB; ++j) rb[d][j] = chunk_settle(rb[d][j], k0 + kc, KB);
        }
#pragma unroll
        for (int j = 0; j < LA; ++j) *(u32x4 *)(smem + slot * SLOT_A + (4 * j + wave) * 1024 + lane * 16) = ra[d][j];
#pragma unroll
        for (int j = 0; j < LB; ++j)
            *(u32x4 *)(smem + B_BASE + slot * SLOT_B + (4 * j + wave) * 1024 + lane * 16) = rb[d][j];
    };

    const int fr = lane & 15, fq = lane >> 4;
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](int slot) __attribute__((always_inline)) {
        const char *sa = smem + slot * SLOT_A + (wm * WTM + fr) * 128;
        const char *sb = smem + B_BASE + slot * SLOT_B + (wn * WTN + fr) * 128;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int c = ((4 * st + fq) ^ swz16(fr)) << 4;
            u32x4 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[i] = *(const u32x4 *)(sa + i * 16 * 128 + c);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[j] = *(const u32x4 *)(sb + j * 16 * 128 + c);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = prod_mfma<T>(fb[j], fa[i], acc[i][j]);
        }
    };

    typename Epi::template Regs<TM, TN> regs;
    const int row0 = m0 + wm * WTM, col0 = n0 + wn * W;
    e.template scales<TM, TN>(regs, lane, row0, col0, p.M, p.N);

    if constexpr (ANY) {
        // tile t's chunks are in registers t % PD until they are written to slot
        // t % 2, before the barrier that opens it; that slot's last reads were
        // before the barrier that opened tile t - 1
        auto step = [&](int t, auto d) __attribute__((always_inline)) {
            constexpr int D = decltype(d)::value;
            write_any(t, D);
            read_any(t + PD, D);                       // (past K: the rows' ends, settled to zeros)
            wait_lgkmcnt0();
            barrier();
            compute(t & 1);
        };
        if (KB >= 16) {
            static_for<0, PD>([&](auto d) { read_any(decltype(d)::value, decltype(d)::value); });
            int t = 0;
            for (; t + PD <= nt; t += PD)
                static_for<0, PD>([&](auto d) __attribute__((always_inline)) { step(t + decltype(d)::value, d); });
            static_for<0, PD - 1>([&](auto d) __attribute__((always_inline)) {
                if (t + decltype(d)::value < nt) step(t + decltype(d)::value, d);
            });
            wait_lgkmcnt0();
            barrier();
        } else if (KB > 0) {                           // rows shorter than a chunk: one tile
            const int kb = group * 128 + kc;
#pragma unroll
            for (int j = 0; j < LA; ++j) ra[0][j] = load_chunk<T>(pa[j], kb, KB);
#pragma unroll
            for (int j = 0; j < LB; ++j) rb[0][j] = load_chunk<T>(pb[j], kb, KB);
            write_any(0, 0);
            wait_lgkmcnt0();
            barrier();
            compute(0);
            wait_lgkmcnt0();
            barrier();
        }
    } else if (nt > 0) {
#pragma unroll
        for (int t = 0; t < S - 1; ++t) fetch(t, t);
        int slot = 0, next = S - 1;
        for (int t = 0; t < nt; ++t) {
            wait_vmcnt<(S - 2) * (LA + LB)>();         // tile t landed
            barrier();                                 // for every wave; and tile t - 1's slot is free
            fetch(t + S - 1, next);
            compute(slot);
            wait_lgkmcnt0();
            next = slot;
            slot = slot + 1 == S ? 0 : slot + 1;
        }
        wait_vmcnt<0>();                               // no load still writes a slot
        barrier();
    }
    if (e.add)
        e.template prepare<TM, TN, false, true>(regs, lane, row0, col0, p.M, p.N);
    if constexpr (KS > 1) {
        // (every wave is past the last reads of the slots)
        if (group > 0) {
            float *sums = (float *)(lds + ((group - 1) * 4 + wave) * SUMS) + lane * 4;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) *(f32x4 *)(sums + (i * TN + j) * 256) = acc[i][j];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int k = 1; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const f32x4 v = *(const f32x4 *)((float *)(lds + ((k - 1) * 4 + wave) * SUMS) + lane * 4 + (i * TN + j) * 256);
                    if constexpr (T == kI8)
                        acc[i][j] = __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, acc[i][j]) + __builtin_bit_cast(i32x4, v));
                    else
                        acc[i][j] += v;
                }
        stage_fence();
    }
    float *stage = (float *)(KS > 1 ? lds + (KS - 1) * 4 * SUMS + wave * STAGE : lds + wave * STAGE);
    if (e.add)
        e.template block<TM, TN, false, false, true>(regs, acc, stage, lane, row0, col0, p.M, p.N);
    else
        e.template block<TM, TN, false, false, false>(regs, acc, stage, lane, row0, col0, p.M, p.N);
}

// QUARTERS: the tiles are the quarters of those 256 x 256 tiles (in prod_w4's
// order) that fill no round of workgroups.
template <int T, int BM, int BN, int S, int KS, bool PAIR, bool ANY, class Epi, bool QUARTERS = false>
__global__ void __launch_bounds__(256 * KS) prod_mid_kernel(ProdArgs p, Epi e) {
    __shared__ __attribute__((aligned(1024))) char lds[kMidLds<BM, BN, S, KS>];
    int tmi, tni;
    if constexpr (QUARTERS) {
        static_assert(BM == 128 && BN == 128, "quarters");
        const int q = blockIdx.x & 3;
        tile_order(p.run + (blockIdx.x >> 2), p.tiles_m * p.tiles_n, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
        tmi = 2 * tmi + (q >> 1), tni = 2 * tni + (q & 1);
        if (tmi * BM >= p.M || tni * (PAIR ? BN / 2 : BN) >= p.N) return;    // (past the matrix's edge)
    } else {
        tile_order(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    }
    prod_mid_body<T, BM, BN, S, KS, PAIR, ANY>(p, tmi, tni, lds, e);
}

// Two products in one launch: the first on workgroups below `split`, the second
// on the others, each with as many as it has tiles.
template <int T, int BM, int BN, int S, int KS, class Epi0, class Epi1>
__global__ void __launch_bounds__(256 * KS) prod_mid_two_kernel(ProdPair q, Epi0 e0, Epi1 e1) {
    __shared__ __attribute__((aligned(1024))) char lds[kMidLds<BM, BN, S, KS>];
    const bool second = (int)blockIdx.x >= q.split;
    const ProdArgs p = second ? q.p[1] : q.p[0];
    const int wg = second ? blockIdx.x - q.split : blockIdx.x;
    int tmi, tni;
    tile_order(wg, p.tiles_m * p.tiles_n, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    if (second)
        prod_mid_body<T, BM, BN, S, KS, false, false>(p, tmi, tni, lds, e1);
    else
        prod_mid_body<T, BM, BN, S, KS, false, false>(p, tmi, tni, lds, e0);
}

}  // namespace tg
