// tree_attn_tc.cu -- attention of a window of drafted tokens over the paged cache on
// the tensor cores (bf16, D = 64, 128 or 256).
//
// A block works through the pieces of its chunk (attn_common.cuh) tile by tile:
//   S = Q K^T     tcgen05.mma kind::f16, 128 query rows x TN keys, fp32 in TMEM
//   P = 2^(S scale log2 e - m), rounded to bf16, back into TMEM over S
//   O += P V      tcgen05.mma kind::f16, P from TMEM, V as it lies in its pages
//                 (token rows of 64-element runs: the MN-major operand), fp32 in TMEM
// One producer warp copies the pages' rows by TMA (one box of min(P, TN) tokens by 64
// dims per lane, the page numbers looked up a tile ahead), one warp issues the
// MMAs, and a warpgroup of 128 threads, one query row each, does each tile's softmax.
// Two arrangements keep the tensor core and the copies busy while a softmax runs:
//   NQ = 1, D <= 128: the tiles of one query tile go to two warpgroups in turn, each
//     with its own S, running maximum and O; the two halves are merged at the end.
//   NQ = 2, D <= 128: windows of more than 128 rows; each warpgroup has a query tile of
//     its own and both use every key/value tile that is copied.
//   NQ = 1, D = 256: O takes half of TMEM, so there is one warpgroup, and S has two
//     buffers of 64 keys, so that the next scores are formed during a softmax.
// The G query heads of a kv head are rows of the same tile, so every key and value is
// copied once for all of them: decoding is bound by HBM as long as a row group is below
// some 280 rows (the machine's products per byte).
//
// The running maximum is only moved when a row's maximum has grown by more than 2^8
// over it: until then the probabilities are taken against the old one, which is exact
// (they and their sum stay below 2^8 times as large, far inside fp32 and bf16's
// range), and O is not read and rescaled.  P is rounded to bf16 because it is an
// operand of the second product; m, l and O are fp32.
//
// Rows of a tile past the last token, which hold whatever the page or the buffer held,
// and drafted tokens with a value that is not finite are zeroed in the V tile before
// the second product, since 0 times NaN is not 0; such a draft's term is added to the
// rows that attend to it at the end.  Only tiles that hold drafted tokens are looked at.
//
// Every wait is bounded.  One that runs out raises the block's abort flag, on which all
// roles leave their loops; the producer then waits for the copies it has in flight and
// the MMA warp for its MMAs, TMEM is freed, and the status word gets TIMEOUT.
#include <mutex>
#include <type_traits>

#include <cuda.h>

#include "attn_common.cuh"
#include "launch_setup.cuh"
#include "ptx_sm100.cuh"

namespace gdnspec {
namespace tat {

constexpr int kRows = 128;               // query rows of an MMA
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 8.0f;            // log2 of what the maximum may grow by before it is moved
constexpr int kSmemMax = 232448;

template <int D, int NQ>
struct Lay {
    static constexpr int TN = D == 256 ? 64 : 128;             // keys of a tile
    static constexpr int NWG = D == 256 ? 1 : 2;               // softmax warpgroups, streams of O
    static constexpr bool kShare = NQ == 2;                    // both streams use every tile
    static constexpr bool kTurns = NWG == 2 && !kShare;        // tiles go to the streams in turn
    static constexpr int kStep = kTurns ? 2 : 1;               // from a stream's tile to its next
    // two warpgroups: a third holds the producer and the MMA warp and gives registers up, so that a softmax thread
    // can hold its row's 128 scores (168 x 384 = 208 x 256 + 88 x 128)
    static constexpr int kThreads = NWG == 2 ? 384 : 192;
    static constexpr int kRegsMore = 208, kRegsLess = 88;
    static constexpr uint32_t kBlocks = D / 64;                // 64-dim blocks of a row
    static constexpr uint32_t kQTile = kRows * D * 2;          // one query tile
    static constexpr int QB = D == 64 ? 2 : 1;                 // buffers of NQ query tiles
    static constexpr uint32_t kStage = TN * D * 2;             // one K or V tile
    // Stages stand in rings, one for each warp that uses them in order: with tiles in turn every stream has its
    // own, so that each stage's barriers are met by the same warps in every phase.
    static constexpr int kRings = kTurns ? 2 : 1;
    static constexpr int NR = D == 64 ? (kTurns ? 5 : 9) : (kTurns ? 3 : 5);
    static constexpr int NST = kRings * NR;
    static constexpr uint32_t kOffKV = QB * NQ * kQTile;
    static constexpr uint32_t kOffMisc = kOffKV + NST * kStage;
    // TMEM columns
    static constexpr uint32_t kColO = 2 * TN > 256 ? 256 : (D == 256 ? 256 : 2 * TN);
    __host__ __device__ static constexpr uint32_t col_s(int i) { return i * TN; }
    __host__ __device__ static constexpr uint32_t col_o(int w) { return kColO + w * D; }
};

// Shared memory behind the tiles.
struct Misc {
    uint64_t full[10], empty[10], q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], pv_done[2], o_full, o_empty, drain[2], clean[2];
    float2 ml[2][kRows];                  // (m, l) of the two streams' rows, exchanged when they are merged
    unsigned long long bad[3];            // drafts whose values are not finite, by piece modulo 3
    int scratch[kAttnScratch];
    uint32_t tmem;
    int abort;
};

// Bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t limit = kWaitLimitDefault) {
    for (uint32_t it = 0; it < limit; ++it) {
        if (ptx::mbar_try_wait(bar, parity, 256u)) return true;
        if ((it & 15u) == 15u && *abort) return false;
    }
    *abort = 1;
    return false;
}

// The same by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                         uint32_t limit = kWaitLimitDefault) {
    return __all_sync(0xffffffffu, wait(bar, parity, abort, limit));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a tcgen05.ld brought is only valid behind its wait: uses depend on this.
template <int N>
__device__ __forceinline__ void landed(uint32_t (&r)[N]) {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void landed32(uint32_t *r) {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Barrier of the softmax warpgroups; whether any thread came with `bad`.
__device__ __forceinline__ bool any_at_barrier(int threads, bool bad) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "bar.red.or.pred q, 1, %1, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(threads), "r"((uint32_t)bad)
        : "memory");
    return r != 0;
}

// Place of tile i's values, of a piece of n tiles, in its ring's order: K V K V .., or, with one stream,
// K0 K1 V0 K2 V1 .. (the next scores are formed before this tile's sums).
template <class L> __device__ __forceinline__ int pos_v(int i, int n) {
    return L::NWG == 2 ? 2 * (i / L::kStep) + 1 : (i < n - 1 ? 2 * i + 2 : 2 * n - 1);
}
// Places that a piece of n tiles takes in ring r.
template <class L> __device__ __forceinline__ int ring_places(int n, int r) {
    return L::kTurns ? 2 * ((n + 1 - r) >> 1) : 2 * n;
}

// Which of a tile's keys a row attends to, as 128 bits: keys before `len` all, drafted
// ones by the row's mask (already cut to the row's tokens).
__device__ __forceinline__ void visible_bits(int k0, int len, uint64_t mask, uint32_t (&bits)[4]) {
    uint64_t lo, hi;
    const int n = len - k0;   // committed keys of the tile
    if (n <= 0) {
        lo = n > -64 ? mask >> -n : 0;
        hi = 0;
    } else if (n < 64) {
        lo = ((1ull << n) - 1) | (mask << n);
        hi = mask >> (64 - n);
    } else {
        lo = ~0ull;
        hi = n == 64 ? mask : n < 128 ? ((1ull << (n - 64)) - 1) | (mask << (n - 64)) : ~0ull;
    }
    bits[0] = (uint32_t)lo;
    bits[1] = (uint32_t)(lo >> 32);
    bits[2] = (uint32_t)hi;
    bits[3] = (uint32_t)(hi >> 32);
}

// ------------------------------------------------------------------ producer warp

template <int D, int NQ>
__device__ __forceinline__ void produce(const AttnArgs &A, const CUtensorMap *mq, const CUtensorMap *mk,
                                        const CUtensorMap *mv, Misc *ms, uint32_t base, const AttnPlan &plan, int group,
                                        int qt, int lane) {
    using L = Lay<D, NQ>;
    const int BR = min(A.C.P, L::TN), chunks = L::TN / BR;    // tokens of a box, boxes of a 64-dim block
    const int my_chunk = lane % chunks, my_blk = lane / chunks;
    const bool mine = my_blk < (int)L::kBlocks;
    const int RT = A.MT / NQ, tokens_q = RT / A.G;             // rows and tokens of a query tile
    const uint32_t box_bytes = BR * 128u;
    const uint32_t q_bytes = 128u * A.G * min(tokens_q, A.T);   // one 64-dim block of one query tile
    uint32_t issued[2] = {0, 0}, q_issued = 0;
    bool ok = true;
    AttnWalk walk = attn_walk(plan, group);
    AttnPiece pc;
    while (ok && walk.next(A, &pc)) {
        if (pc.cnt * A.G - qt * A.MT <= 0) continue;
        const int kv = pc.len + pc.cnt, n = pc.t1 - pc.t0;
        const int32_t *table = A.C.page_table + (int64_t)pc.slot * A.C.max_pages;
        // row of the pool where this lane's box of tile t starts, -1: no token of it is in use
        const auto box_row = [&](int t) {
            const int64_t tok = (int64_t)t * L::TN + my_chunk * BR;
            if (!mine || t >= pc.t1 || tok >= kv) return -1;
            int page = table[tok >> A.C.logP];
            if (page < 0 || page >= A.C.num_pages) {
                atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
                page = 0;
            }
            return ((A.layer * A.C.num_pages + page) * A.C.HKV + pc.h) * A.C.P + ((int)tok & (A.C.P - 1));
        };
        const auto copy = [&](const CUtensorMap *map, int row, int t) {
            const int r = L::kTurns ? (t - pc.t0) & 1 : 0;
            const uint32_t p = r ? issued[1] : issued[0], st = r * L::NR + p % L::NR, ph = (p / L::NR) & 1u;
            if (!all_wait(ptx::smem_addr(&ms->empty[st]), ph ^ 1u, &ms->abort)) return false;
            const uint32_t bar = ptx::smem_addr(&ms->full[st]);
            const int left = kv - t * L::TN, live = min(chunks, (left + BR - 1) / BR);
            if (lane == 0) ptx::mbar_expect_tx(bar, box_bytes * live * L::kBlocks);
            __syncwarp();
            if (row >= 0)
                ptx::tma_load_2d(base + L::kOffKV + st * L::kStage + my_blk * (L::TN * 128u) + my_chunk * box_bytes, map,
                                 bar, my_blk * 64, row);
            if (r) ++issued[1]; else ++issued[0];
            return true;
        };
        int row = box_row(pc.t0), next = box_row(pc.t0 + 1);
        ok = copy(mk, row, pc.t0);
        if (ok) {   // the query tiles, behind the first keys
            const uint32_t qb = q_issued % L::QB, ph = (q_issued / L::QB) & 1u;
            ok = all_wait(ptx::smem_addr(&ms->q_empty[qb]), ph ^ 1u, &ms->abort);
            if (ok) {
                const uint32_t bar = ptx::smem_addr(&ms->q_full[qb]);
                const int t0 = qt * NQ * tokens_q;
                int tiles = 0;
#pragma unroll
                for (int s = 0; s < NQ; ++s) tiles += t0 + s * tokens_q < pc.cnt;
                if (lane == 0) ptx::mbar_expect_tx(bar, q_bytes * L::kBlocks * tiles);
                __syncwarp();
                if (lane < (int)L::kBlocks * tiles) {
                    const int s = lane / L::kBlocks, blk = lane - s * L::kBlocks;
                    ptx::tma_load_3d(base + (qb * NQ + s) * L::kQTile + blk * (kRows * 128u), mq, bar, blk * 64,
                                     pc.h * A.G, pc.b * A.T + t0 + s * tokens_q);
                }
                ++q_issued;
            }
        }
        if (ok && !L::kShare && n > 1) ok = copy(mk, next, pc.t0 + 1);
        for (int i = 0; ok && i < n; ++i) {   // values of tile i, then the keys that are used after them
            const int t = pc.t0 + i;
            const int after = box_row(t + 2);
            ok = copy(mv, row, t);
            if (L::kShare) {
                if (ok && i + 1 < n) ok = copy(mk, next, t + 1);
            } else {
                if (ok && i + 2 < n) ok = copy(mk, after, t + 2);
            }
            row = next;
            next = after;
        }
    }
    if (!ok) {   // copies in flight land before the block's shared memory goes away
        for (int r = 0; r < L::kRings; ++r)
            for (uint32_t p = issued[r] > L::NR ? issued[r] - L::NR : 0; p < issued[r]; ++p)
                ptx::mbar_wait(ptx::smem_addr(&ms->full[r * L::NR + p % L::NR]), (p / L::NR) & 1u);
        for (uint32_t p = q_issued > L::QB ? q_issued - L::QB : 0; p < q_issued; ++p)
            ptx::mbar_wait(ptx::smem_addr(&ms->q_full[p % L::QB]), (p / L::QB) & 1u);
    }
}

// ------------------------------------------------------------------ MMA warp

// A value that all lanes hold, from one of them: the tensor core's operands are uniform
// registers, and values that come from memory or from a loop are only seen to be
// uniform behind a shuffle (without it each MMA costs some 300 cycles to issue).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Stream w of the block: with two streams each has a warp of its own, so that one's wait for a softmax does not
// hold up the other's products.
template <int D, int NQ>
__device__ __forceinline__ void multiply(const AttnArgs &A, Misc *ms, uint32_t base, uint32_t tmem, const AttnPlan &plan,
                                         int group, int qt, int w) {
    using L = Lay<D, NQ>;
    constexpr uint32_t idesc_s = ptx::idesc_bf16(kRows, L::TN);
    constexpr uint32_t idesc_o = ptx::idesc_bf16(kRows, D) | ptx::kIdescBMn;
    const int ring = L::kTurns ? w * L::NR : 0;   // first stage of this warp's ring
    const uint32_t d_o = uniform(tmem + L::col_o(w));
    uint32_t q_used = 0, pieces = 0;
    uint32_t c_ph = 0;                          // bit of a barrier: parity of the waits done on clean
    uint32_t p_ph = 0, pv_ph = 0, pv_any = 0;   // bit of a buffer: parity of the waits done on p_full, of the commits
                                                // made on pv_done, whether there was one
    bool ok = true;
    const auto bar = [](uint64_t &b) { return ptx::smem_addr(&b); };
    // Everything that a product needs is made uniform before the wait that it hangs on, so that nothing but the
    // issue lies between the two.
    struct Stage {
        uint32_t at, ph;   // stage of the ring, parity of its phase
    };
    const auto after = [](Stage s, int n) {
        s.at += n;
        if (s.at >= (uint32_t)L::NR) {
            s.at -= L::NR;
            s.ph ^= 1u;
        }
        return s;
    };
    struct Op {
        uint64_t a, b;
        uint32_t p, empty, full, ph;
    };
    const auto op = [&](Stage s, bool values, uint32_t q_addr, int buf) {
        Op o;
        const uint32_t addr = uniform(base + L::kOffKV + (ring + s.at) * L::kStage);
        o.a = ptx::smem_desc_sw128(uniform(q_addr));
        o.b = values ? ptx::smem_desc_sw128_mn(addr, L::TN * 128u) : ptx::smem_desc_sw128(addr);
        o.p = uniform(tmem + L::col_s(buf));
        o.empty = uniform(bar(ms->empty[ring + s.at]));
        o.full = bar(ms->full[ring + s.at]);
        o.ph = s.ph;
        return o;
    };
    const auto wait_full = [&](const Op &o) { return all_wait(o.full, o.ph, &ms->abort, A.wait_limit); };
    // S of a buffer = query tile times K tile
    const auto scores = [&](const Op &o, int buf, bool last) {
        const uint32_t done = uniform(bar(ms->s_full[buf])), q_done = uniform(bar(ms->q_empty[q_used % L::QB]));
        ptx::tc_fence_after_sync();
        if (ptx::elect_one()) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)   // descriptors count in 16 bytes
                ptx::mma_bf16(o.p, o.a + ((ks >> 2) * (kRows * 128u) + (ks & 3) * 32u) / 16,
                              o.b + ((ks >> 2) * (L::TN * 128u) + (ks & 3) * 32u) / 16, idesc_s, ks != 0);
            ptx::mma_commit(done);
            ptx::mma_commit(o.empty);
            if (last) ptx::mma_commit(q_done);
        }
        __syncwarp();
    };
    // O of this stream (+)= steps [K0, K1) of P times the V tile
    const auto sums = [&](const Op &o, int buf, auto k0, auto k1, uint32_t keep) {
        constexpr int K0 = decltype(k0)::value, K1 = decltype(k1)::value;
        const uint32_t done = uniform(bar(ms->pv_done[buf]));
        ptx::tc_fence_after_sync();
        if (ptx::elect_one()) {
#pragma unroll
            for (int ks = K0; ks < K1; ++ks)
                ptx::mma_bf16_tmem_a(d_o, o.p + ks * 8, o.b + ks * 2048u / 16, idesc_o, ks != 0 ? 1u : keep);
            if (K1 == L::TN / 16) {
                ptx::mma_commit(done);
                ptx::mma_commit(o.empty);
            }
        }
        __syncwarp();
        if (K1 == L::TN / 16) {
            pv_ph ^= 1u << buf;
            pv_any |= 1u << buf;
        }
    };
    const auto commit = [&](uint64_t &b) {
        if (ptx::elect_one()) ptx::mma_commit(bar(b));
        __syncwarp();
    };
    // S buffer `buf` may be written again once the sums that read its P are done
    const auto wait_free = [&](int buf) {
        return !((pv_any >> buf) & 1u) || all_wait(bar(ms->pv_done[buf]), ((pv_ph >> buf) & 1u) ^ 1u, &ms->abort);
    };
    using Zero = std::integral_constant<int, 0>;
    using Half = std::integral_constant<int, L::TN / 32>;
    using All = std::integral_constant<int, L::TN / 16>;
    Stage sk = {0, 0}, sv = {0, 0};   // of the next K and V tile
    AttnWalk walk = attn_walk(plan, group);
    AttnPiece pc;
    bool any = walk.next(A, &pc);
    if (w == 0 && qt == 0 && ptx::elect_one()) attn_note(A, group, any, pc, plan.chunk);
    __syncwarp();
    for (; ok && any; any = walk.next(A, &pc)) {
        if (pc.cnt * A.G - qt * A.MT <= 0) continue;
        const int n = pc.t1 - pc.t0;
        const uint32_t qb = q_used % L::QB;
        const uint32_t q_addr = base + (qb * NQ + (L::kShare ? w : 0)) * L::kQTile;
        const auto o_free = [&] { return all_wait(bar(ms->o_empty), (pieces & 1u) ^ 1u, &ms->abort); };
        ok = all_wait(bar(ms->q_full[qb]), (q_used / L::QB) & 1u, &ms->abort, A.wait_limit);
        if (L::NWG == 2) {
            // one S buffer a stream: scores, softmax, sums, then the next scores over what the sums have read
            const int first = L::kTurns ? w : 0;
            for (int i = first; ok && i < n; i += L::kStep) {
                const Op qk = op(sk, false, q_addr, w);
                ok = wait_full(qk) && wait_free(w);
                if (!ok) break;
                scores(qk, w, i + L::kStep >= n);
                sv = after(sk, 1);
                sk = after(sk, 2);
                const Op pv = op(sv, true, q_addr, w);
                const uint32_t keep = uniform(i > first);
                const uint32_t half = bar(ms->p_half[w]), full = bar(ms->p_full[w]), ph = p_ph & 1u;
                p_ph ^= 1u;
                ok = wait_full(pv) && (i > first || o_free());
                if (L::kShare && w == 1) {
                    // a shared tile with drafts is cleaned by the first warpgroup: the window lies in at most two tiles
                    const int d = pc.t0 + i - pc.len / L::TN;
                    if (d >= 0) {
                        ok = ok && all_wait(bar(ms->clean[d]), (c_ph >> d) & 1u, &ms->abort);
                        c_ph ^= 1u << d;
                    }
                }
                ok = ok && all_wait(half, ph, &ms->abort);
                if (!ok) break;
                sums(pv, w, Zero(), Half(), keep);
                ok = all_wait(full, ph, &ms->abort);
                if (!ok) break;
                sums(pv, w, Half(), All(), 1u);
            }
            if (ok && first >= n) {   // no tile for this stream; every phase of o_empty is waited for all the same
                commit(ms->q_empty[qb]);
                ok = o_free();
            }
        } else {
            // two S buffers: the next scores are formed before this tile's sums; the ring goes K0 K1 V0 K2 V1 ..
            Op qk = op(sk, false, q_addr, 0);
            ok = ok && wait_full(qk) && wait_free(0);
            if (ok) scores(qk, 0, n == 1);
            sk = after(sk, 1);
            for (int i = 0; ok && i < n; ++i) {
                const int buf = i & 1;
                if (i + 1 < n) {
                    qk = op(sk, false, q_addr, buf ^ 1);
                    ok = wait_full(qk) && wait_free(buf ^ 1);
                    if (!ok) break;
                    scores(qk, buf ^ 1, i + 2 == n);
                    sk = after(sk, 1);
                }
                const Op pv = op(sk, true, q_addr, buf);
                sk = after(sk, 1);
                const uint32_t keep = uniform(i > 0);
                const uint32_t ph = (p_ph >> buf) & 1u;
                p_ph ^= 1u << buf;
                ok = wait_full(pv) && (i || o_free()) && all_wait(bar(ms->p_full[buf]), ph, &ms->abort);
                if (!ok) break;
                sums(pv, buf, Zero(), All(), keep);
            }
        }
        if (ok) commit(ms->o_full);
        ++q_used;
        ++pieces;
    }
    if (!ok) {   // no MMA is running when TMEM is freed
        commit(ms->drain[w]);
        ptx::mbar_wait(bar(ms->drain[w]), 0);
    }
}

// ------------------------------------------------------------------ softmax

// Rows of a V tile that the second product must not see: past the last token, and
// drafts that are not finite, which go into *bad.  By the 128 threads of a warpgroup.
template <int D, int NQ>
__device__ __forceinline__ void clean_values(uint8_t *tile, int k0, int len, int kv, int tid, unsigned long long *bad) {
    using L = Lay<D, NQ>;
    constexpr int kPieces = D / 8;   // 16-byte pieces of a row
    const int first = max(len - k0, 0);
    unsigned long long mine = 0;
    for (int i = first * kPieces + tid; i < L::TN * kPieces; i += 128) {
        const int r = i / kPieces, c = i - r * kPieces;
        uint4 *p = reinterpret_cast<uint4 *>(tile + (c >> 3) * (L::TN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        if (k0 + r >= kv) {
            *p = make_uint4(0, 0, 0, 0);
        } else {
            const uint4 x = *p;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u) mine |= 1ull << (k0 + r - len);
        }
    }
    if (mine) atomicOr(bad, mine);
    asm volatile("bar.sync %0, 128;" ::"r"(2 + (int)(threadIdx.x >> 7)) : "memory");
    const unsigned long long all = *reinterpret_cast<volatile unsigned long long *>(bad);
    if (all)
        for (int i = first * kPieces + tid; i < min(L::TN, kv - k0) * kPieces; i += 128) {
            const int r = i / kPieces, c = i - r * kPieces;
            if ((all >> (k0 + r - len)) & 1)
                *reinterpret_cast<uint4 *>(tile + (c >> 3) * (L::TN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(0, 0, 0, 0);
        }
    ptx::fence_proxy_async_smem();
}

// The terms of drafts that are not finite, for the rows that attend to them: weight
// and value from memory.  o: dims d0 .. d0 + 31 of this row's unnormalised sums over m.
__device__ __noinline__ void add_bad(const AttnArgs &A, const AttnPiece &pc, unsigned long long bad, int64_t qrow, float m,
                                     int d0, float *o) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(A.q) + qrow * A.C.D;
    while (bad) {
        const int j = __ffsll((long long)bad) - 1;
        bad &= bad - 1;
        const int64_t row = kv_token_row(A.C, pc.slot, pc.len + j);
        if (row < 0) continue;
        const int64_t e = kv_elem(A.C, A.layer, pc.h, row);
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(A.C.k) + e, *v = static_cast<const __nv_bfloat16 *>(A.C.v) + e;
        float s = 0.0f;
        for (int d = 0; d < A.C.D; ++d) s = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), s);
        const float p = __bfloat162float(__float2bfloat16_rn(ex2(s * A.scale_log2 - m)));
        for (int d = 0; d < 32; ++d) o[d] = fmaf(p, __bfloat162float(v[d0 + d]), o[d]);
    }
}

template <int D, int NQ>
__device__ __forceinline__ void soften(const AttnArgs &A, Misc *ms, uint8_t *sm, uint32_t tmem, const AttnPlan &plan,
                                       int group, int qt, int tid_all) {
    using L = Lay<D, NQ>;
    constexpr int kBothThreads = L::NWG * 128;
    const int w = tid_all >> 7, tid = tid_all & 127, warp = tid >> 5;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    const int RT = A.MT / NQ;
    const int my_row = (L::kShare ? w * RT : 0) + tid;      // row of the block's MT
    const float c = A.scale_log2;
    const auto bar = [](uint64_t &b) { return ptx::smem_addr(&b); };
    uint32_t used = 0, pieces = 0;
    uint32_t s_ph = 0, pv_ph = 0;                           // bit of a buffer: parity of the tiles taken, handed on
    bool ok = true;
    AttnWalk walk = attn_walk(plan, group);
    AttnPiece pc;
    while (ok && walk.next(A, &pc)) {
        const int live = min(A.MT, pc.cnt * A.G - qt * A.MT);
        if (live <= 0) continue;
        const int n = pc.t1 - pc.t0, kv = pc.len + pc.cnt;
        const bool on = tid < RT && my_row < live;
        const bool warp_on = __any_sync(0xffffffffu, on);
        const int r = qt * A.MT + my_row;
        uint64_t mask = 0;
        if (on) {
            mask = attn_mask(A, pc.b, r / A.G);
            if (pc.cnt < 64) mask &= (1ull << pc.cnt) - 1;
        }
        float m = -INFINITY, l = 0.0f;
        // A thread whose wait ran out goes on without waiting or computing, so that the warpgroup's barriers are
        // met by all, until the barrier at the piece's end tells everybody.
        const int first = L::kTurns ? w : 0;
        for (int i = first; i < n; i += L::kStep) {
            const int buf = L::NWG == 2 ? w : i & 1, o = w;
            const bool drafts = (pc.t0 + i + 1) * L::TN > pc.len;   // the tile holds drafted tokens, or ends the row
            const int k0 = (pc.t0 + i) * L::TN;
            ok = __all_sync(0xffffffffu, ok && wait(bar(ms->s_full[buf]), (s_ph >> buf) & 1u, &ms->abort));
            s_ph ^= 1u << buf;
            ptx::tc_fence_after_sync();
            const bool ok_half = ok;
            if (ok && warp_on) {
                // eight chains of three-input maxima (one chain's latency would be the whole row's), taken of each 32
                // scores while the next are on their way from TMEM
                uint32_t s[L::TN];
                float tops[8];
                uint32_t bits[4];
                if (drafts) visible_bits(k0, pc.len, mask, bits);
                ptx::tmem_ld32_bits(lane_addr + L::col_s(buf), s);
#pragma unroll
                for (int x = 0; x < L::TN; x += 32) {
                    landed32(s + x);
                    if (x + 32 < L::TN) ptx::tmem_ld32_bits(lane_addr + L::col_s(buf) + x + 32, s + x + 32);
                    if (drafts) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((bits[x >> 5] >> j) & 1u)) s[x + j] = 0xff800000u;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = __uint_as_float(s[x + j]), b = __uint_as_float(s[x + 8 + j]);
                        const float d = __uint_as_float(s[x + 16 + j]), e = __uint_as_float(s[x + 24 + j]);
                        tops[j] = x == 0 ? max3(a, b, d) : max3(max3(tops[j], a, b), d, e);
                        if (x == 0) tops[j] = fmaxf(tops[j], e);
                    }
                }
                const float top = c * max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]),
                                           fmaxf(tops[6], tops[7]));
                const bool move = top > m + kGrow || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, move)) {
                    const float to = move ? top : m;
                    const float al = m == -INFINITY ? 0.0f : ex2(m - to);
                    l *= al;
                    m = to;
                    if (i > first) {
                        // the sums so far, in O, are those of the stream's tile before this one
                        if (L::NWG == 1)
                            ok = __all_sync(0xffffffffu, wait(bar(ms->pv_done[buf ^ 1]), ((pv_ph >> (buf ^ 1)) & 1u) ^ 1u,
                                                              &ms->abort));
                        if (ok) {
                            ptx::tc_fence_after_sync();
#pragma unroll 1
                            for (int x = 0; x < D; x += 8) {   // few at a time: the row's scores are held as well
                                uint32_t u[8];
                                ptx::tmem_ld8_bits(lane_addr + L::col_o(o) + x, u);
                                landed(u);
#pragma unroll
                                for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * al);
                                ptx::tmem_st8_bits(lane_addr + L::col_o(o) + x, u);
                            }
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.0f : -m;
                const uint64_t c2 = pair(c, c), off2 = pair(off, off);
                uint64_t sum[4] = {0, 0, 0, 0};   // pairs of zeros
#pragma unroll
                for (int x = 0; x < L::TN; x += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(s[x + 2 * j]), __uint_as_float(s[x + 2 * j + 1])), c2, off2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[j & 3] = add2(sum[j & 3], pair(a, b));
                        p[j] = pack_bf16(a, b);
                    }
                    ptx::tmem_st16_bits(lane_addr + L::col_s(buf) + x / 2, p);
                    if (L::NWG == 2 && x + 32 == L::TN / 2 && !drafts) {   // the sums begin on the first half
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if ((tid & 31) == 0) ptx::mbar_arrive(bar(ms->p_half[buf]));
                    }
                }
                float s0, s1;
                unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                l += s0 + s1;
                ptx::tmem_st_wait();
            }
            if (drafts && (!L::kShare || w == 0)) {
                const uint32_t pos = used + pos_v<L>(i, n), st = (L::kTurns ? w * L::NR : 0) + pos % L::NR;
                ok = __all_sync(0xffffffffu, ok && wait(bar(ms->full[st]), (pos / L::NR) & 1u, &ms->abort));
                clean_values<D, NQ>(sm + L::kOffKV + st * L::kStage, k0, pc.len, kv, tid, &ms->bad[pieces % 3]);
                if (L::kShare) {
                    __syncwarp();
                    if ((tid & 31) == 0) ptx::mbar_arrive(bar(ms->clean[pc.t0 + i - pc.len / L::TN]));
                }
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if ((tid & 31) == 0) {
                if (L::NWG == 2 && (drafts || !(ok_half && warp_on))) ptx::mbar_arrive(bar(ms->p_half[buf]));
                ptx::mbar_arrive(bar(ms->p_full[buf]));
            }
            pv_ph ^= 1u << buf;
        }
        ok = ok && wait(bar(ms->o_full), pieces & 1u, &ms->abort);
        ptx::tc_fence_after_sync();
        // ---- the piece's rows: merge the streams, put out or keep
        if (L::kTurns) ms->ml[w][tid] = make_float2(m, l);
        if (tid_all == 0) ms->bad[(pieces + 1) % 3] = 0;
        ok = !any_at_barrier(kBothThreads, !ok);
        float w0 = 1.0f, w1 = 0.0f;
        if (L::kTurns) {
            const float2 a = ms->ml[0][tid], b = ms->ml[1][tid];
            m = fmaxf(a.x, b.x);
            w0 = a.y == 0.0f ? 0.0f : ex2(a.x - m);
            w1 = b.y == 0.0f ? 0.0f : ex2(b.x - m);
            l = a.y * w0 + b.y * w1;
        }
        unsigned long long bad = ms->bad[pieces % 3] & mask;
        if (ok && warp_on) {
            const int64_t row = attn_out_row(A, pc.b, pc.h, on ? r : qt * A.MT);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            // the two warpgroups of a shared query tile take half of the dims each
            constexpr int kDims = L::kTurns ? D / 2 : D;
            const int d_begin = L::kTurns ? w * kDims : 0;
            const int64_t part = (int64_t)blockIdx.x * 2 + pc.side;
            const bool whole = pc.whole();
#pragma unroll 1
            for (int x = 0; x < kDims; x += 32) {
                const int d0 = d_begin + x;
                float f[32];
                if (L::kTurns) {
                    uint32_t u[32], v[32];
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(0) + d0, u);
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(1) + d0, v);
                    landed(u);
                    landed(v);
#pragma unroll
                    for (int j = 0; j < 32; ++j)   // a stream that saw nothing may hold anything
                        f[j] = (w0 != 0.0f ? __uint_as_float(u[j]) * w0 : 0.0f) +
                               (w1 != 0.0f ? __uint_as_float(v[j]) * w1 : 0.0f);
                } else {
                    uint32_t u[32];
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(L::kShare ? w : 0) + d0, u);
                    landed(u);
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = l != 0.0f ? __uint_as_float(u[j]) : 0.0f;
                }
                if (on) {
                    if (bad) {   // rare: a copy of its own, so that f stays in registers
                        float g[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = f[j];
                        add_bad(A, pc, bad, row, m, d0, g);
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = g[j];
                    }
                    if (whole) {
                        uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(A.out) + row * D + d0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            out[j] = make_uint4(pack_bf16(f[8 * j] * inv, f[8 * j + 1] * inv),
                                                pack_bf16(f[8 * j + 2] * inv, f[8 * j + 3] * inv),
                                                pack_bf16(f[8 * j + 4] * inv, f[8 * j + 5] * inv),
                                                pack_bf16(f[8 * j + 6] * inv, f[8 * j + 7] * inv));
                    } else {
                        float4 *po = A.part_o + (part * (D / 4) + d0 / 4) * A.MT + my_row;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            po[(int64_t)j * A.MT] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
                    }
                }
            }
            if (on && d_begin == 0) {
                if (!whole) A.part_ml[part * A.MT + my_row] = make_float2(m, l);
                else if (A.lse) A.lse[row] = attn_lse(m, l);
            }
        }
        ptx::tc_fence_before_sync();
        __syncwarp();
        if ((tid & 31) == 0) ptx::mbar_arrive(bar(ms->o_empty));
        used += ring_places<L>(n, w);
        ++pieces;
    }
}

template <int D, int NQ>
__global__ void __launch_bounds__(Lay<D, NQ>::kThreads, 1)
tree_attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs A) {
    using L = Lay<D, NQ>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *sm = smem_raw + pad;
    Misc *ms = reinterpret_cast<Misc *>(sm + L::kOffMisc);
    const uint32_t base = raw + pad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = blockIdx.x / A.NQT, qt = blockIdx.x - group * A.NQT;
    uint32_t have;
    asm("mov.u32 %0, %dynamic_smem_size;" : "=r"(have));
    if (pad + L::kOffMisc + sizeof(Misc) > have) {   // the segment does not start where it always has
        if (tid == 0) atomicOr(A.C.status, GDN_SPEC_ST_TIMEOUT);
        return;
    }
    if (tid == 0) {
        const auto init = [](uint64_t &b, uint32_t n) { ptx::mbar_init(ptx::smem_addr(&b), n); };
        for (int i = 0; i < L::NST; ++i) {
            init(ms->full[i], 1);
            init(ms->empty[i], NQ);            // streams that use a tile
        }
        for (int i = 0; i < 2; ++i) {
            init(ms->q_full[i], 1);
            init(ms->q_empty[i], L::NWG);
            init(ms->s_full[i], 1);
            init(ms->p_half[i], 4);
            init(ms->p_full[i], 4);
            init(ms->pv_done[i], 1);
        }
        init(ms->o_full, L::NWG);
        init(ms->o_empty, L::NWG * 4);
        for (int i = 0; i < 2; ++i) {
            init(ms->drain[i], 1);
            init(ms->clean[i], 4);
        }
        ms->bad[0] = ms->bad[1] = ms->bad[2] = 0;
        ms->abort = 0;
        ptx::mbar_init_fence();
        ptx::prefetch_tmap(&mq);
        ptx::prefetch_tmap(&mk);
        ptx::prefetch_tmap(&mv);
    }
    if (warp == 0) ptx::tmem_alloc(ptx::smem_addr(&ms->tmem), kTmemCols);
    grid_dep_wait();   // nothing in global memory was touched so far
    attn_dead_rows<__nv_bfloat16>(A, blockIdx.x, gridDim.x, L::kThreads);
    const AttnPlan plan = attn_plan<L::kThreads>(A, group, blockIdx.x == 0, ms->scratch);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;

    if (warp < L::NWG * 4) {
        if (L::NWG == 2) more_registers<L::kRegsMore>();
        soften<D, NQ>(A, ms, sm, tmem, plan, group, qt, tid);
    } else {
        if (L::NWG == 2) fewer_registers<L::kRegsLess>();
        if (warp == L::NWG * 4) produce<D, NQ>(A, &mq, &mk, &mv, ms, base, plan, group, qt, lane);
        if (warp > L::NWG * 4 && warp <= L::NWG * 5) multiply<D, NQ>(A, ms, base, tmem, plan, group, qt, warp - L::NWG * 4 - 1);
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && ms->abort) atomicOr(A.C.status, GDN_SPEC_ST_TIMEOUT);
    grid_dep_launch();
}

// ------------------------------------------------------------------ host

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// bf16 tensor of `rank` dims, the innermost `dims[0]` dense; strides in elements.
bool bf16_map(CUtensorMap *map, const void *p, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
              const cuuint32_t *box) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t bytes[3];
    cuuint32_t one[3] = {1, 1, 1};
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] * 2;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(p), dims, bytes, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NQ>
cudaError_t run(const AttnArgs &A, cudaStream_t st) {
    using L = Lay<D, NQ>;
    static_assert(L::kOffMisc + sizeof(Misc) <= kSmemMax, "shared memory");
    // room to reach a 1024-byte boundary (the dynamic segment starts on one: there is no static one)
    constexpr size_t need = L::kOffMisc + sizeof(Misc) + 1024;
    constexpr size_t smem = need < (size_t)kSmemMax ? need : (size_t)kSmemMax;
    static KernelSetup setup;
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)tree_attn_tc_kernel<D, NQ>, smem, &sms);
    if (e != cudaSuccess) return e;
    const cuuint64_t rows = (cuuint64_t)A.C.n_layers * A.C.num_pages * A.C.HKV * A.C.P;
    const cuuint64_t kv_dims[2] = {(cuuint64_t)D, rows}, kv_stride[1] = {(cuuint64_t)D};
    const cuuint32_t kv_box[2] = {64, (cuuint32_t)(A.C.P < L::TN ? A.C.P : L::TN)};
    const int tokens_q = A.MT / NQ / A.G;
    const cuuint64_t q_dims[3] = {(cuuint64_t)D, (cuuint64_t)A.HQ, (cuuint64_t)A.B * A.T};
    const cuuint64_t q_stride[2] = {(cuuint64_t)D, (cuuint64_t)A.HQ * D};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)A.G, (cuuint32_t)(tokens_q < A.T ? tokens_q : A.T)};
    CUtensorMap mq, mk, mv;
    if (!bf16_map(&mk, A.C.k, 2, kv_dims, kv_stride, kv_box) || !bf16_map(&mv, A.C.v, 2, kv_dims, kv_stride, kv_box) ||
        !bf16_map(&mq, A.q, 3, q_dims, q_stride, q_box))
        return cudaErrorInvalidValue;
    return launch_dependent(tree_attn_tc_kernel<D, NQ>, dim3(A.groups * A.NQT), dim3(L::kThreads), smem, st, mq, mk, mv, A);
}

}  // namespace tat

bool tree_attn_tc_supported(const KvArgs &C, int G, bool bf16) {
    return bf16 && (C.D == 64 || C.D == 128 || C.D == 256) && G <= tat::kRows &&
           (int64_t)C.n_layers * C.num_pages * C.HKV * C.P <= INT32_MAX;
}

// The cut of the work: a query tile holds whole tokens, as many as fit in 128 rows;
// windows beyond one tile take two side by side where TMEM holds both (D <= 128).
void tree_attn_tc_cut(AttnArgs *A, int sms) {
    const int R = A->T * A->G, tile = tat::kRows / A->G * A->G;
    const int nq = A->C.D <= 128 && R > tile ? 2 : 1;
    A->TN = A->C.D == 256 ? 64 : 128;
    A->MT = nq * tile;
    A->NQT = (R + A->MT - 1) / A->MT;
    const int groups = sms / A->NQT;
    A->groups = groups < 1 ? 1 : groups;
    A->min_chunk = 1;
}

cudaError_t launch_tree_attn_tc(const AttnArgs &A, cudaStream_t st) {
    const bool two = A.MT > tat::kRows;
    cudaError_t e;
    if (A.C.D == 64) e = two ? tat::run<64, 2>(A, st) : tat::run<64, 1>(A, st);
    else if (A.C.D == 128) e = two ? tat::run<128, 2>(A, st) : tat::run<128, 1>(A, st);
    else e = tat::run<256, 1>(A, st);
    return e != cudaSuccess ? e : launch_attn_join(A, true, st);
}

}  // namespace gdnspec
