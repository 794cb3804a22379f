// Products in 256 x 256 tiles (PAIR: 256 rows and 128 gated columns), for
// grids that fill the GPU: one persistent workgroup per CU of four waves, each
// with a 128 x 128 quadrant as 8 x 8 blocks of 16 x 16 accumulators in AGPRs.
//
// K tiles of 128 bytes in two LDS slots an operand.  A wave issues 128 MFMAs a
// K tile in two steps of 64 bytes; the second step of tile t - 1 runs after the
// barrier that opens tile t, so that the matrix pipe does not drain there:
//   after barrier t:  64 MFMAs of tile t - 1 step 1, between them the fragment
//                     reads of tile t step 0 and the loads of tile t + 1
//                     64 MFMAs of tile t step 0, between them the reads of
//                     tile t step 1
//                     wait for the loads; barrier t + 1
// After a tile's last K step the next tile's first loads are issued, into the
// slots K tile 0 always uses, and then the finished tile's results are staged
// and stored from the last slots.
//
// A K tile takes 1.37 to 1.41 us (MFMAs busy 71 to 83 % of the cycles, 61 % where
// K is short for the results, int8 8192 x 14336 x 4096; LDS three quarters of
// them): int8 8192^3 373 to 407 us, 2.7 to 2.95 POP/s, bf16 8192 x 4096 x 28672
// 1.57 PFLOP/s.
//
// Grids of one round at most run the same schedule in tiles of 256 x 128 and 128
// x 128 (TN 4; TM 8 and 4) with three and four slots: a K tile's MFMAs take half
// the time and a quarter of it, so its loads are issued two and three K tiles
// ahead (256 x 128: two slots 0.86 us a K tile with 160 workgroups, three 0.73).
#pragma once

#include "prod.hpp"

namespace tg {

// acc = a.b + acc, or a.b, in place in AGPRs.
template <int T, bool ZERO>
__device__ __forceinline__ void prod_mfma_agpr(f32x4 &acc, const u32x4 &a, const u32x4 &b) {
#define TG_PROD_MFMA(op)                                                                         \
    if constexpr (ZERO)                                                                          \
        asm volatile(op " %0, %1, %2, 0" : "=a"(acc) : "v"(a), "v"(b));                          \
    else                                                                                         \
        asm volatile(op " %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b))
    if constexpr (T == kI8) {
        TG_PROD_MFMA("v_mfma_i32_16x16x64_i8");
    } else if constexpr (T == 2) {
        TG_PROD_MFMA("v_mfma_f32_16x16x32_f16");
    } else {
        TG_PROD_MFMA("v_mfma_f32_16x16x32_bf16");
    }
#undef TG_PROD_MFMA
}

// The last MFMAs' results are in their registers behind this (a 16x16 one's 8
// passes and the longest wait that a read of its result needs: 36 cycles).
template <int TM, int TN>
__device__ __forceinline__ void prod_result_fence(f32x4 (&acc)[TM][TN]) {
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 3" : "+a"(acc[0][0]), "+a"(acc[0][1]), "+a"(acc[0][2]), "+a"(acc[0][3]));
#pragma unroll
    for (int k = 4; k < TM * TN; k += 4) {
        f32x4 *a = &acc[k / TN][k % TN];
        asm volatile("" : "+a"(a[0]), "+a"(a[1]), "+a"(a[2]), "+a"(a[3]));
    }
}

// LDS of a workgroup with 16 TN rows of B a wave (TN 8 as above; 4: 256 x 128
// tiles, PAIR 64 columns): slots of K tiles, and what lines brought ahead leave
// behind.
template <int TM, int TN> constexpr int kW4Slots = TN == 8 ? 2 : TM == 8 ? 3 : 4;
template <int TM, int TN> constexpr int kW4Lds = kW4Slots<TM, TN> * 32 * (TM + TN) * 128 + 1024;

// Workgroup wg of nwg that walk the tiles wg, wg + nwg, ... below p.run.
// reload(): p again, from memory; prepare(lane, row0, col0, M, N) loads what a
// quadrant's results need, before the tile's last MFMAs and the next one's first
// loads; emit(regs, acc, stage, lane, row0, col0, M, N) stores them and waits for
// all that was issued before their last stores.  (Operand rows on 16 bytes, KB > 0 a multiple of 16.)
template <int T, bool PAIR, bool PREFETCH, int TM, int TN, class Reload, class Prepare, class Emit>
__device__ __forceinline__ void prod_w4_body(const ProdArgs &p, int wg, int nwg, char *smem, Reload &&reload,
                                             Prepare &&prepare, Emit &&emit) {
    constexpr int Q = TM * TN, SLOT = 32 * TM * 128, B_SLOT = 32 * TN * 128;
    constexpr int NS = kW4Slots<TM, TN>, B_BASE = NS * SLOT, LOADS = TM + TN;
    constexpr int BM = 32 * TM;
    constexpr int BN = PAIR ? 16 * TN : 32 * TN;       // result columns of a tile
    constexpr int W = BN / 2, STAGE = 16 * kStagePitch<W> * 4;
    // K tile t brings the lines of tile t + PF; NS - 2 tiles' come ahead of the loop, behind tile PF0
    constexpr int PF = NS + 1, PF0 = PF - (NS - 2) - 1;
    static_assert((TM == 8 && TN == 8) || TN == 4, "schedule");
    static_assert(2 * STAGE <= B_SLOT && 2 * STAGE <= SLOT && kW4Lds<TM, TN> == B_BASE + NS * B_SLOT + 1024, "LDS");

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int vt = wg, tmi, tni;
    tile_order(vt, p.tiles_m * p.tiles_n, p.tiles_m, p.tiles_n, p.group_m, tmi, tni);
    int m0 = tmi * BM, n0 = tni * BN;
    const int KB = p.KB, nt = (KB + 127) / 128;

    // Load instruction j of a wave: A rows 32 j + 8 wave + lane / 8, B the same
    // or (PAIR) rows 16 j + 8 (wave % 2) + lane / 8 of the wave's half.  Lane l
    // writes chunk l % 8 and fetches chunk (l % 8) ^ (l / 8); the K offset goes
    // with the lane's offset (beyond the resource for a chunk past K, which
    // then reads as zeros), 32 or 16 rows with the scalar one.
    const bool up = PAIR && wave >= 2;
    const int64_t ldb = up ? p.ldb1 : p.ldb;
    const int kc = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t aoff = (uint32_t)((8 * wave + (lane >> 3)) * p.lda) + kc;
    const uint32_t boff = (uint32_t)(((PAIR ? 8 * (wave & 1) : 8 * wave) + (lane >> 3)) * ldb) + kc;
    const int astep = (int)(32 * p.lda), bstep = (int)((PAIR ? 16 : 32) * ldb);
    __amdgpu_buffer_rsrc_t rA, rB;
    auto resources = [&](const ProdArgs &a) __attribute__((always_inline)) {
        const int64_t lb = up ? a.ldb1 : a.ldb;
        rA = make_rsrc((const char *)a.A + (int64_t)m0 * a.lda, span_bytes(a.M - m0, a.KB, a.lda, 1));
        rB = make_rsrc((const char *)(up ? a.B1 : a.B) + (int64_t)n0 * lb, span_bytes(a.N - n0, a.KB, lb, 1));
    };
    resources(p);
    auto dma = [&](__amdgpu_buffer_rsrc_t r, int lds, uint32_t voff, int soff) __attribute__((always_inline)) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(smem + lds), 16, voff,
                                                 soff, 0, 0);
    };
    // The K tiles are taken in a circle that starts at another place on each of
    // the 8 XCDs: with rows a multiple of 4 KiB apart, a K tile's chunks of all
    // rows lie in few memory channels, and the XCDs would meet there (gated 8192
    // x 14336 x 4096: 1342 us, 1446 in step).
    const int k_first = (wg & 7) * nt / 8 * 128;
    auto koff = [&](int t) __attribute__((always_inline)) {
        const int k = t * 128 + k_first;
        return t >= nt ? KB : k >= nt * 128 ? k - nt * 128 : k;
    };
    // (into slot s: K tile t's is t % 2, a constant in the loop unrolled by two)
    auto fetch_a = [&](int t, int s, int j) __attribute__((always_inline)) {
        const int k0 = koff(t);
        const uint32_t v = k0 + kc < KB ? aoff + k0 : kOOB;
        dma(rA, s * SLOT + (4 * j + wave) * 1024, v, j * astep);
    };
    auto fetch_b = [&](int t, int s, int j) __attribute__((always_inline)) {
        const int k0 = koff(t);
        const uint32_t v = k0 + kc < KB ? boff + k0 : kOOB;
        dma(rB, B_BASE + s * B_SLOT + (4 * j + wave) * 1024, v, j * bstep);
    };

    // Lines of K tile t + PF brought into this XCD's L2, a 128-byte line a lane:
    // of each of its panels a workgroup takes the part that falls to it among
    // those that share the panel (in the tile order 8 share rows of A and 4 rows
    // of B), an eighth of A's rows and a quarter of B's.  Four bytes of each line go to LDS that
    // nobody reads; the wait at a window's end leaves them in flight.  Hides
    // what the L2s miss (gradients of 8192 x 14336 x 4096: 3280 -> 3020 us; 2 or
    // 5 tiles ahead the same).
    auto pf_off = [&]() __attribute__((always_inline)) {
        if (wave == 0) return lane < BM / 8 ? (uint32_t)((BM / 8 * (tni & 7) + lane) * (int)p.lda) : kOOB;
        constexpr int OF_B = PAIR ? 4 * TN : 8 * TN;
        return wave < (PAIR ? 3 : 2) && lane < OF_B ? (uint32_t)((OF_B * (tmi & 3) + lane) * (int)ldb) : kOOB;
    };
    uint32_t pfo = pf_off();
    int pfk = 0;                                       // K offset of the tile next prefetched
    auto prefetch = [&]() __attribute__((always_inline)) {
        pfk = pfk + 128 >= nt * 128 ? pfk + 128 - nt * 128 : pfk + 128;    // (past the end: the circle again)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wave == 0 ? rA : rB, (__attribute__((address_space(3))) void *)(smem + B_BASE + NS * B_SLOT + wave * 256), 4, pfo, pfk, 0, 0);
    };

    const int fr = lane & 15, fq = lane >> 4, fswz = swz16(fr);
    int a_read[2], b_read[2];                          // [step]
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        a_read[st] = (wm * 16 * TM + fr) * 128 + (((4 * st + fq) ^ fswz) << 4);
        b_read[st] = B_BASE + (wn * 16 * TN + fr) * 128 + (((4 * st + fq) ^ fswz) << 4);
    }
    f32x4 acc[TM][TN];
    u32x4 fa[2][TM], fb[2][TN];                        // [step][block]
    // fragment read k of step st from slot s, in the order the MFMAs use them: A
    // block 0, the B blocks, the other A blocks
    auto read_frag = [&](int s, int st, int k) __attribute__((always_inline)) {
        if (k == 0 || k > TN) {
            const int i = k == 0 ? 0 : k - TN;
            fa[st][i] = *(const u32x4 *)(smem + a_read[st] + (s * SLOT + i * 16 * 128));
        } else {
            fb[st][k - 1] = *(const u32x4 *)(smem + b_read[st] + (s * B_SLOT + (k - 1) * 16 * 128));
        }
    };
    auto mfma = [&](auto zero, int st, int i, int j) __attribute__((always_inline)) {
        prod_mfma_agpr<T, decltype(zero)::value>(acc[i][j], fb[st][j], fa[st][i]);
        __builtin_amdgcn_sched_barrier(0);
    };
    // One K tile, in slot S, the one NS - 1 ahead into the last one's; FIRST: none before it (accumulators start from zero).
    auto tile = [&](auto first, auto slot, int t) __attribute__((always_inline)) {
        constexpr int S = decltype(slot)::value, FREE = (S + NS - 1) % NS;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (!decltype(first)::value) mfma(std::false_type(), 1, q / TN, q % TN);
            if constexpr (TN == 8) {
                if (q % 4 == 0) read_frag(S, 0, q / 4);
                if (q % 8 == 0) fetch_a(t + NS - 1, FREE, q / 8);
                if (q % 8 == 4) fetch_b(t + NS - 1, FREE, q / 8);
            } else {
                if (q % 2 == 0 && q / 2 < TM + TN) read_frag(S, 0, q / 2);
                if (q % 4 == 1) fetch_a(t + NS - 1, FREE, q / 4);
                if (q % TM == 3) fetch_b(t + NS - 1, FREE, q / TM);
            }
            if (PREFETCH && q == Q - 1) prefetch();
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            mfma(first, 0, q / TN, q % TN);
            constexpr int EVERY = TN == 8 ? 3 : TM == 8 ? 2 : 1;
            if (q % EVERY == 0 && q / EVERY < TM + TN) read_frag(S, 1, q / EVERY);
        }
        // tile t + 1 landed; what was issued behind its loads may be on its way
        wait_vmcnt<(NS - 2) * LOADS + (PREFETCH ? NS - 1 : 0)>();
        wait_lgkmcnt0();
        barrier();
    };

    // (in the order of the loop: a K tile's lines behind the loads of another)
    pfk = (k_first + PF0 * 128) % (nt * 128);
    static_for<0, NS - 1>([&](auto t) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TM; ++j) fetch_a(t, t, j);
#pragma unroll
        for (int j = 0; j < TN; ++j) fetch_b(t, t, j);
        if (PREFETCH && t > 0) prefetch();
    });
    wait_vmcnt<(NS - 2) * (LOADS + (PREFETCH ? 1 : 0))>();
    barrier();
    float *stage = (float *)(smem + (wave < 2 ? (NS - 1) * SLOT : B_BASE + (NS - 1) * B_SLOT) + (wave & 1) * STAGE);
    while (true) {
        tile(std::true_type(), std::integral_constant<int, 0>(), 0);
        int t = 1;
        for (; t + NS - 1 < nt; t += NS)
            static_for<0, NS>([&](auto k) __attribute__((always_inline)) {
                tile(std::false_type(), std::integral_constant<int, (k + 1) % NS>(), t + k);
            });
        static_for<0, NS - 1>([&](auto k) __attribute__((always_inline)) {
            if (t + k < nt) tile(std::false_type(), std::integral_constant<int, (k + 1) % NS>(), t + k);
        });
        const ProdArgs r = reload();
        const int dm0 = m0, dn0 = n0;
        auto regs = prepare(lane, dm0 + wm * 16 * TM, dn0 + wn * W, r.M, r.N);
#pragma unroll
        for (int q = 0; q < Q; ++q) mfma(std::false_type(), 1, q / TN, q % TN);
        prod_result_fence<TM, TN>(acc);
        // (every wave is past its last barrier, so past all reads of the slots;
        // the loads of the tiles past the end have landed there)
        if constexpr (NS > 2) {
            wait_vmcnt<0>();
            barrier();
        }
        vt += nwg;
        const bool more = vt < r.run;
        if (more) {
            tile_order(vt, r.tiles_m * r.tiles_n, r.tiles_m, r.tiles_n, r.group_m, tmi, tni);
            m0 = tmi * BM;
            n0 = tni * BN;
            resources(r);
            pfo = pf_off();
            int wv = wave;                             // (their LDS addresses are computed here, not held)
            asm volatile("" : "+s"(wv));
            pfk = (k_first + PF0 * 128) % (nt * 128);
            static_for<0, NS - 1>([&](auto t) __attribute__((always_inline)) {
                const int k0 = koff(t);
                const uint32_t va = k0 + kc < KB ? aoff + k0 : kOOB, vb = k0 + kc < KB ? boff + k0 : kOOB;
#pragma unroll
                for (int j = 0; j < TM; ++j) dma(rA, t * SLOT + (4 * j + wv) * 1024, va, j * astep);
#pragma unroll
                for (int j = 0; j < TN; ++j) dma(rB, B_BASE + t * B_SLOT + (4 * j + wv) * 1024, vb, j * bstep);
                if (PREFETCH && t > 0) prefetch();
            });
        }
        emit(regs, acc, stage, lane, dm0 + wm * 16 * TM, dn0 + wn * W, r.M, r.N);
        if (!more) {
            wait_vmcnt<0>();
            break;
        }
        wait_lgkmcnt0();
        barrier();
    }
}

template <class Epi, int TM, int TN>
__device__ __forceinline__ void prepare_agpr(const Epi &e, typename Epi::template Regs<TM, TN> &regs, int lane, int row0,
                                             int col0, int M, int N) {
    e.template scales<TM, TN>(regs, lane, row0, col0, M, N);
    with_form(e, [&](auto vec, auto add) __attribute__((always_inline)) {
        e.template prepare<TM, TN, vec, add>(regs, lane, row0, col0, M, N);
    });
}

// An epilogue's results.  The next tile's first loads have landed then; the
// results' stores issued after them, of which there are at least stores(), may
// still run.
template <class Epi, int TM, int TN>
__device__ __forceinline__ void emit_agpr(const Epi &e, typename Epi::template Regs<TM, TN> &regs, const f32x4 (&acc)[TM][TN],
                                          float *stage, int lane, int row0, int col0, int M, int N) {
    with_form(e, [&](auto vec, auto add) __attribute__((always_inline)) {
        e.template block<TM, TN, true, vec, add>(regs, acc, stage, lane, row0, col0, M, N);
        wait_vmcnt<vec ? Epi::template stores<TM, TN>() : 0>();
    });
}

template <int T, bool PAIR, bool PREFETCH, class Epi, int TN = 8, int TM = 8>
__global__ void __launch_bounds__(256) prod_w4_kernel(ProdArgs p, Epi e) {
    __shared__ __attribute__((aligned(1024))) char smem[kW4Lds<TM, TN>];
    typedef typename Epi::template Regs<TM, TN> Regs;
    prod_w4_body<T, PAIR, PREFETCH, TM, TN>(
        p, blockIdx.x, gridDim.x, smem, [] { return kernel_arg0_reloaded<ProdArgs>(); },
        [&](int lane, int row0, int col0, int M, int N) __attribute__((always_inline)) {
            Regs r;
            prepare_agpr<Epi, TM, TN>(e, r, lane, row0, col0, M, N);
            return r;
        },
        [&](Regs &regs, const auto &acc, float *stage, int lane, int row0, int col0, int M, int N)
            __attribute__((always_inline)) { emit_agpr(e, regs, acc, stage, lane, row0, col0, M, N); });
}

// Two products in one launch: the first on workgroups below `split`, the second
// on the others, each in rounds of its own.
template <int T, class Epi0, class Epi1>
__global__ void __launch_bounds__(256) prod_w4_two_kernel(ProdPair q, Epi0 e0, Epi1 e1) {
    __shared__ __attribute__((aligned(1024))) char smem[kW4Lds<8, 8>];
    const bool second = (int)blockIdx.x >= q.split;
    const ProdArgs p = second ? q.p[1] : q.p[0];
    const int wg = second ? blockIdx.x - q.split : blockIdx.x;
    if (wg >= p.run) return;                           // (more workgroups than tiles)
    struct Regs {
        typename Epi0::template Regs<8, 8> a;
        typename Epi1::template Regs<8, 8> b;
    };
    prod_w4_body<T, false, true, 8, 8>(
        p, wg, second ? gridDim.x - q.split : q.split, smem,
        [&]() __attribute__((always_inline)) {
            const ProdPair r = kernel_arg0_reloaded<ProdPair>();
            return second ? r.p[1] : r.p[0];
        },
        [&](int lane, int row0, int col0, int M, int N) __attribute__((always_inline)) {
            Regs r;
            if (second)
                prepare_agpr<Epi1, 8, 8>(e1, r.b, lane, row0, col0, M, N);
            else
                prepare_agpr<Epi0, 8, 8>(e0, r.a, lane, row0, col0, M, N);
            return r;
        },
        [&](Regs &regs, const auto &acc, float *stage, int lane, int row0, int col0, int M, int N) __attribute__((always_inline)) {
            if (second)
                emit_agpr(e1, regs.b, acc, stage, lane, row0, col0, M, N);
            else
                emit_agpr(e0, regs.a, acc, stage, lane, row0, col0, M, N);
        });
}

}  // namespace tg
