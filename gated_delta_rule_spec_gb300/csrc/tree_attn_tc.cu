// tree_attn_tc.cu -- attention of a window of drafted tokens over the paged cache on
// the tensor cores (bf16; heads of other than 64, 128 or 256 dims are filled up with
// zeros to the next of them in shared memory).
//
// A block works through the pieces of its chunk (attn_common.cuh) in tiles of 64 keys:
//   S = Q K^T     tcgen05.mma kind::f16, 128 query rows x 64 keys, fp32 in TMEM
//   P = 2^(S scale log2 e - m), rounded to bf16, back into TMEM over S
//   O += P V      tcgen05.mma kind::f16, P from TMEM, V as it lies in its pages
//                 (token rows of 64-element runs: the MN-major operand), fp32 in TMEM
// The tiles go through one or two streams.  A stream is a warpgroup of 128 threads, one
// query row each, for the softmax, two buffers of S in TMEM, so that its next scores
// are formed while a softmax runs, and an O that stays in TMEM over the piece.
//   NQ = 1, D <= 128: one query tile; its key/value tiles go to the two streams in turn,
//     each with a running maximum and an O of its own, merged at the end.
//   NQ = 2, D <= 128: windows of more than 128 rows; each stream has a query tile of
//     its own and both use every key/value tile that is copied.
//   NQ = 1, D = 256: O takes half of TMEM, so there is one stream.
// One producer warp copies the pages' rows by TMA, two tiles to a stage where D <= 128
// (boxes of min(P, 64) tokens; all of a tile's dims by one copy where a page holds the
// tile), and the products are issued by warps of their own, first and second ones
// apart: a wait on a barrier costs some 150 cycles even where it is ready, and an issue
// blocks while the tensor core is busy, so one warp that issued both products of a
// tile took longer than its softmax (32 rows of 64 drafts over up to 8192 tokens, 64
// heads on 8 of 128: 466 us; with tiles of 128 keys and one buffer of S, where scores,
// softmax and sums wait for one another, 492 us; as it is 333 us when the same call is
// replayed, 0.53 of the bf16 rate, and 349 to 352 us in calls on changing inputs).
// There the first product bounds it: an MMA of 128 x 64 takes as long as one of
// 128 x 128, because the query rows come from shared memory.
// The G query heads of a kv head are rows of the same tile, so every key and value is
// copied once for all of them, and with fewer rows the copies are the bound: 4 rows of
// 131072 tokens, 32 heads on 8 of 128: 251 to 255 us, 0.97 to 0.99 of the copy bandwidth;
// 128 rows of 8 drafts over up to 4096 tokens, 16 heads on 2 of 256: 128 to 130 us, 0.82.
//
// The running maximum is only moved when a row's maximum has grown by more than 2^8
// over it, an idea published for attention kernels of this generation: until then the probabilities are taken against the old one, which is exact
// (they and their sum stay below 2^8 times as large, far inside fp32 and bf16's
// range), and O is not read and rescaled.  P is rounded to bf16 because it is an
// operand of the second product; m, l and O are fp32, and l is the sum of the values
// before that rounding, so that lse keeps fp32's accuracy (out is off by 0.0023 of
// itself against 64 bits, where its own rounding alone is 0.0017).
//
// Rows of a tile past the last token, which hold whatever the page or the buffer held,
// and drafted tokens with a value that is not finite are zeroed in the V tile before
// the second product, since 0 times NaN is not 0; such a draft's term is added to the
// rows that attend to it at the end.  Only tiles that hold drafted tokens are looked at.
// Where two streams share a tile the first one cleans it; the warp that issues the sums
// takes the first stream's before the second's.
//
// Every wait is bounded.  One that runs out raises the block's abort flag, on which all
// roles leave their loops; the producer then waits for the copies it has in flight and
// the MMA warp for its MMAs, TMEM is freed, and the status word gets TIMEOUT.
#include <type_traits>

#include "attn_common.cuh"
#include "attn_tc.cuh"
#include "launch_setup.cuh"

namespace gdnspec {
namespace tat {

constexpr int kRows = 128;               // query rows of an MMA
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemMax = 232448;

constexpr int kTile = 64;                // keys of a tile
constexpr int kMaxStages = 12;

template <int D, int NQ>
struct Lay {
    static constexpr int NWG = D == 256 ? 1 : 2;               // streams
    static constexpr bool kShare = NQ == 2;                    // both streams use every tile
    static constexpr bool kTurns = NWG == 2 && !kShare;        // units of tiles go to the streams in turn
    static constexpr int kThreads = NWG == 2 ? 384 : 256;      // softmax warpgroups; producer and MMA warps
    static constexpr int kUnit = D == 256 ? 1 : 2;             // tiles that are copied together, one stage
    static constexpr uint32_t kBlocks = D / 64;                // 64-dim blocks of a row
    static constexpr uint32_t kBlock = kTile * 128;            // one of them, of a tile
    static constexpr uint32_t kQTile = kRows * D * 2;          // one query tile
    static constexpr int QB = D == 64 ? 2 : 1;                 // buffers of NQ query tiles
    static constexpr uint32_t kStage = kUnit * kTile * D * 2;
    // Stages stand in rings: one for the keys and one for each user of values (with units in turn each stream has its
    // own), so that a stage's barriers are met by the same warps in every phase.
    static constexpr int NK = D == 64 ? 4 : 2;
    static constexpr int NV = D == 64 ? (kTurns ? 4 : 6) : kTurns ? 2 : 3;
    static constexpr int kRings = kTurns ? 3 : 2;
    static constexpr int NST = NK + (kRings - 1) * NV;
    static constexpr uint32_t kOffKV = QB * NQ * kQTile;
    static constexpr uint32_t kOffMisc = kOffKV + NST * kStage;
    __host__ __device__ static constexpr int ring_of(int w) { return kTurns ? 1 + w : 1; }   // a stream's values
    __host__ __device__ static constexpr int first(int ring) { return ring ? NK + (ring - 1) * NV : 0; }
    __host__ __device__ static constexpr int size(int ring) { return ring ? NV : NK; }
    // TMEM columns: four buffers of S, then O
    __host__ __device__ static constexpr uint32_t col_s(int w, int buf) { return (2 * w + buf) * kTile; }
    __host__ __device__ static constexpr uint32_t col_o(int w) { return 256 + w * D; }
};

// Shared memory behind the tiles.
struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages], q_full[2], q_empty[2];
    uint64_t s_full[4], p_full[4], pv_done[4];   // by stream and buffer of S
    uint64_t o_full, o_empty, drain[3];
    float2 ml[2][kRows];                  // (m, l) of the two streams' rows, exchanged when they are merged
    unsigned long long bad[3];            // drafts whose values are not finite, by piece modulo 3
    int scratch[kAttnScratch];
    uint32_t tmem;
    int abort;
};

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

// Tiles of a piece of n that stream w takes, and which tile of the piece its j-th is.
template <class L> __device__ __forceinline__ int stream_tiles(int n, int w) {
    if (!L::kTurns) return n;
    const int whole = n >> 2, rest = n & 3;   // units of two tiles, w's and the other's
    return 2 * whole + (w ? max(rest - 2, 0) : min(rest, 2));
}
template <class L> __device__ __forceinline__ int stream_tile(int j, int w) {
    return L::kTurns ? 4 * (j >> 1) + 2 * w + (j & 1) : j;
}

// Which of a tile's keys a row attends to, as 64 bits: keys before `len` all, drafted
// ones by the row's mask (already cut to the row's tokens).
__device__ __forceinline__ uint64_t visible_bits(int k0, int len, uint64_t mask) {
    const int n = len - k0;   // committed keys of the tile
    if (n <= 0) return n > -64 ? mask >> -n : 0;
    return n < 64 ? ((1ull << n) - 1) | (mask << n) : ~0ull;
}

// ------------------------------------------------------------------ producer warp

// One lane issues: a copy's operands are uniform registers, and lanes with copies of their own would be served one
// after another.  The lanes look up the pages of a unit's boxes side by side.
template <int D, int NQ>
__device__ __forceinline__ void produce(const AttnArgs &A, const CUtensorMap *mq, const CUtensorMap *mk,
                                        const CUtensorMap *mv, Misc *ms, uint32_t base, const AttnPlan &plan, int group,
                                        int qt) {
    using L = Lay<D, NQ>;
    const int lane = threadIdx.x & 31;
    const int log_br = min(A.C.logP, 6), BR = 1 << log_br;     // tokens of a box: within a page and within a tile
    const int RT = A.MT / NQ, tokens_q = RT / A.G;             // rows and tokens of a query tile
    const uint32_t q_bytes = 128u * A.G * min(tokens_q, A.T);   // one 64-dim block of one query tile
    Place place[3];
    uint32_t issued[3] = {0, 0, 0}, q_issued = 0;
    bool ok = true;
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    while (ok && walk.next(A, &pc)) {
        if (pc.cnt * A.G - qt * A.MT <= 0) continue;
        const int kv = pc.len + pc.cnt, n = pc.t1 - pc.t0;
        const int32_t *table = A.C.page_table + (int64_t)pc.slot * A.C.max_pages;
        const int units = (n + L::kUnit - 1) / L::kUnit;
        // Tokens of unit u of the piece that lie before the end, and the page of its box `lane`.  A page is looked up
        // some units before it is used, so that the table's latency is not waited for.
        const auto live_of = [&](int u) {
            return min(min(L::kUnit, n - u * L::kUnit) * kTile, kv - (pc.t0 + u * L::kUnit) * kTile);
        };
        const auto page_of = [&](int u) {
            return u < units && lane * BR < live_of(u) ? table[((pc.t0 + u * L::kUnit) * kTile + lane * BR) >> A.C.logP] : 0;
        };
        const auto copy = [&](const CUtensorMap *map, auto ring_c, int u, int page) {
            constexpr int ring = decltype(ring_c)::value;
            const uint32_t st = L::first(ring) + place[ring].at;
            const int tok = (pc.t0 + u * L::kUnit) * kTile, boxes = (live_of(u) + BR - 1) >> log_br;
            if (lane < boxes && (page < 0 || page >= A.C.num_pages)) {
                atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
                page = 0;
            }
            // row of the pool where box `lane` starts
            const int row = ((A.layer * A.C.num_pages + page) * A.C.HKV + pc.h) * A.C.P + ((tok + lane * BR) & (A.C.P - 1));
            if (!wait(ptx::smem_addr(&ms->empty[st]), place[ring].ph ^ 1u, &ms->abort)) return false;
            const uint32_t bar = uniform(ptx::smem_addr(&ms->full[st]));
            const uint32_t dst = uniform(base + L::kOffKV + st * L::kStage);
            if (A.whole) {   // all of a tile's blocks by one copy
                int rows[L::kUnit];
#pragma unroll
                for (int c = 0; c < L::kUnit; ++c) rows[c] = __shfl_sync(0xffffffffu, row, c);
                if (ptx::elect_one()) {
                    ptx::mbar_expect_tx(bar, L::kBlocks * L::kBlock * boxes);
#pragma unroll
                    for (int c = 0; c < L::kUnit; ++c)
                        if (c < boxes) ptx::tma_load_3d(dst + c * L::kBlocks * L::kBlock, map, bar, 0, rows[c], 0);
                }
            } else {
                constexpr int kMost = L::kUnit * kTile / 16;   // boxes of the smallest pages
                int rows[kMost];
#pragma unroll
                for (int c = 0; c < kMost; ++c) rows[c] = __shfl_sync(0xffffffffu, row, c);
                if (ptx::elect_one()) {
                    ptx::mbar_expect_tx(bar, BR * 128u * L::kBlocks * boxes);
#pragma unroll
                    for (int c = 0; c < kMost; ++c) {
                        if (c >= boxes) break;
                        const int at = c * BR;   // row of the unit
                        const uint32_t to = dst + (at / kTile) * L::kBlocks * L::kBlock + (at % kTile) * 128u;
#pragma unroll
                        for (int blk = 0; blk < (int)L::kBlocks; ++blk)
                            ptx::tma_load_3d(to + blk * L::kBlock, map, bar, blk * 64, rows[c], 0);
                    }
                }
            }
            __syncwarp();
            ++issued[ring];
            place[ring].step(L::size(ring));
            return true;
        };
        const auto copy_k = [&](int u, int page) { return copy(mk, std::integral_constant<int, 0>(), u, page); };
        const auto copy_v = [&](int u, int page) {
            return L::kTurns && (u & 1) ? copy(mv, std::integral_constant<int, L::kRings - 1>(), u, page)
                                        : copy(mv, std::integral_constant<int, 1>(), u, page);
        };
        int pages[4] = {page_of(0), page_of(1), page_of(2), 0};   // of units u .. u + 3
        ok = copy_k(0, pages[0]);
        if (ok) {   // the query tiles, behind the first keys
            const uint32_t qb = q_issued % L::QB, ph = (q_issued / L::QB) & 1u;
            ok = wait(ptx::smem_addr(&ms->q_empty[qb]), ph ^ 1u, &ms->abort);
            if (ok) {
                const uint32_t bar = uniform(ptx::smem_addr(&ms->q_full[qb]));
                const uint32_t dst = uniform(base + qb * NQ * L::kQTile);
                const int t0 = qt * NQ * tokens_q;
                if (ptx::elect_one()) {
                    int tiles = 0;
#pragma unroll
                    for (int s = 0; s < NQ; ++s) tiles += t0 + s * tokens_q < pc.cnt;
                    ptx::mbar_expect_tx(bar, q_bytes * L::kBlocks * tiles);
                    for (int s = 0; s < tiles; ++s)
#pragma unroll
                        for (int blk = 0; blk < (int)L::kBlocks; ++blk)
                            ptx::tma_load_3d(dst + s * L::kQTile + blk * (kRows * 128u), mq, bar, blk * 64, pc.h * A.G,
                                             pc.b * A.T + t0 + s * tokens_q);
                }
                __syncwarp();
                ++q_issued;
            }
        }
        if (ok && units > 1) ok = copy_k(1, pages[1]);
        for (int u = 0; ok && u < units; ++u) {   // the keys run ahead of the values by two units
            pages[3] = page_of(u + 3);
            ok = copy_v(u, pages[0]);
            if (ok && u + 2 < units) ok = copy_k(u + 2, pages[2]);
#pragma unroll
            for (int x = 0; x < 3; ++x) pages[x] = pages[x + 1];
        }
    }
    if (!ok) {   // copies in flight land before the block's shared memory goes away
#pragma unroll
        for (int r = 0; r < L::kRings; ++r)
            for (uint32_t size = L::size(r), p = issued[r] > size ? issued[r] - size : 0; p < issued[r]; ++p)
                ptx::mbar_wait(ptx::smem_addr(&ms->full[L::first(r) + p % size]), (p / size) & 1u);
        for (uint32_t p = q_issued > L::QB ? q_issued - L::QB : 0; p < q_issued; ++p)
            ptx::mbar_wait(ptx::smem_addr(&ms->q_full[p % L::QB]), (p / L::QB) & 1u);
    }
}

// ------------------------------------------------------------------ MMA warps

// When a warp gives up, none of its MMAs is running when TMEM is freed.
__device__ __forceinline__ void drain(Misc *ms, int who) {
    commit(ptx::smem_addr(&ms->drain[who]));
    ptx::mbar_wait(ptx::smem_addr(&ms->drain[who]), 0);
}

// The first products, S = Q K^T: of stream w where the streams share tiles (an issue
// blocks while the tensor core is busy, and one warp for both streams left it idle
// during its waits), else of all streams.  What an MMA needs is made uniform before
// the wait that it hangs on, so that only the issue is behind it.
template <int D, int NQ>
__device__ __forceinline__ void multiply_scores(const AttnArgs &A, Misc *ms, uint32_t base, uint32_t tmem,
                                                const AttnPlan &plan, int group, int qt, int w) {
    using L = Lay<D, NQ>;
    constexpr uint32_t idesc = ptx::idesc_bf16(kRows, kTile);
    const auto bar = [](uint64_t &b) { return ptx::smem_addr(&b); };
    uint32_t q_used = 0, used_any = 0, used_ph = 0;   // bit of an S buffer: whether it was used, parity of its uses
    Place key;
    bool ok = true;
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    bool any = walk.next(A, &pc);
    if (qt == 0 && w == 0 && ptx::elect_one()) attn_note(A, group, any, pc, plan.chunk);
    __syncwarp();
    for (; ok && any; any = walk.next(A, &pc)) {
        if (pc.cnt * A.G - qt * A.MT <= 0) continue;
        const int n = pc.t1 - pc.t0;
        const uint32_t qb = q_used % L::QB, q_addr = base + (qb * NQ + (L::kShare ? w : 0)) * L::kQTile;
        ok = wait(bar(ms->q_full[qb]), (q_used / L::QB) & 1u, &ms->abort, A.wait_limit);
        for (int i = 0; ok && i < n; i += L::kUnit) {
            const uint32_t keys = uniform(base + L::kOffKV + key.at * L::kStage);
            const uint32_t empty = uniform(bar(ms->empty[key.at])), q_done = uniform(bar(ms->q_empty[qb]));
            ok = wait(bar(ms->full[key.at]), key.ph, &ms->abort, A.wait_limit);
            key.step(L::NK);
#pragma unroll
            for (int t = 0; t < L::kUnit; ++t) {   // the unit's tiles
                const int stream = L::kTurns ? (i >> 1) & 1 : w;
                const int x = 2 * stream + (L::kUnit == 2 ? t : i & 1);   // S buffer
                const bool here = i + t < n, last = i + L::kUnit >= n;
                const uint64_t a = ptx::smem_desc_sw128(uniform(q_addr));
                const uint64_t b = ptx::smem_desc_sw128(keys + t * L::kBlocks * L::kBlock);
                const uint32_t d = uniform(tmem + x * kTile), done = uniform(bar(ms->s_full[x]));
                // the buffer is free once the sums that read its last P are done
                if (ok && here && ((used_any >> x) & 1u))
                    ok = wait(bar(ms->pv_done[x]), ((used_ph >> x) & 1u) ^ 1u, &ms->abort);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    if (here) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)   // descriptors count in 16 bytes
                            ptx::mma_bf16(d, a + ((ks >> 2) * (kRows * 128u) + (ks & 3) * 32u) / 16,
                                          b + ((ks >> 2) * L::kBlock + (ks & 3) * 32u) / 16, idesc, ks != 0);
                        ptx::mma_commit(done);
                    }
                    if (t == L::kUnit - 1) {
                        ptx::mma_commit(empty);
                        if (last) ptx::mma_commit(q_done);
                    }
                }
                __syncwarp();
                if (here) {
                    used_any |= 1u << x;
                    used_ph ^= 1u << x;
                }
            }
        }
        ++q_used;
    }
    if (!ok) drain(ms, w);
}

// The second products, O += P V, of stream w, or of both where they share tiles.
template <int D, int NQ>
__device__ __forceinline__ void multiply_sums(const AttnArgs &A, Misc *ms, uint32_t base, uint32_t tmem,
                                              const AttnPlan &plan, int group, int qt, int w) {
    using L = Lay<D, NQ>;
    constexpr uint32_t idesc = ptx::idesc_bf16(kRows, D) | ptx::kIdescBMn;
    const auto bar = [](uint64_t &b) { return ptx::smem_addr(&b); };
    const int first = L::first(L::ring_of(w));
    uint32_t pieces = 0, p_ph = 0;   // bit of a buffer: parity of the waits done on p_full
    Place val;
    bool ok = true;
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    while (ok && walk.next(A, &pc)) {
        if (pc.cnt * A.G - qt * A.MT <= 0) continue;
        const int mine = stream_tiles<L>(pc.t1 - pc.t0, w);
        const auto o_free = [&] { return wait(bar(ms->o_empty), (pieces & 1u) ^ 1u, &ms->abort); };
        if (mine == 0) ok = o_free();   // every phase is waited for
        for (int j = 0; ok && j < mine; ++j) {
            const int st = first + val.at;
            const int half = j & (L::kUnit - 1);   // tile of the unit
            const bool end = half == L::kUnit - 1 || j == mine - 1;
            const uint64_t b = ptx::smem_desc_sw128_mn(
                uniform(base + L::kOffKV + st * L::kStage + half * L::kBlocks * L::kBlock), L::kBlock);
            const uint32_t keep = uniform(j > 0), empty = uniform(bar(ms->empty[st]));
            if (half == 0) ok = wait(bar(ms->full[st]), val.ph, &ms->abort, A.wait_limit) && (j || o_free());
            if (end) val.step(L::NV);
#pragma unroll
            for (int s = 0; s < NQ; ++s) {
                const int stream = L::kShare ? s : w, x = 2 * stream + (j & 1);
                const uint32_t d = uniform(tmem + L::col_o(stream)), p = uniform(tmem + x * kTile);
                const uint32_t done = uniform(bar(ms->pv_done[x]));
                // (a shared tile with drafts is cleaned by the first warpgroup before it hands its P on)
                ok = ok && wait(bar(ms->p_full[x]), (p_ph >> x) & 1u, &ms->abort);
                p_ph ^= 1u << x;
                if (!ok) break;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks)
                        ptx::mma_bf16_tmem_a(d, p + ks * 8, b + ks * 2048u / 16, idesc, ks != 0 ? 1u : keep);
                    ptx::mma_commit(done);
                    if (end && s == NQ - 1) ptx::mma_commit(empty);
                }
                __syncwarp();
            }
        }
        if (ok) commit(bar(ms->o_full));
        ++pieces;
    }
    if (!ok) drain(ms, 1 + w + (L::kShare ? 1 : 0));
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
    for (int i = first * kPieces + tid; i < kTile * kPieces; i += 128) {
        const int r = i / kPieces, c = i - r * kPieces;
        uint4 *p = reinterpret_cast<uint4 *>(tile + (c >> 3) * (L::kBlock) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
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
        for (int i = first * kPieces + tid; i < min(kTile, kv - k0) * kPieces; i += 128) {
            const int r = i / kPieces, c = i - r * kPieces;
            if ((all >> (k0 + r - len)) & 1)
                *reinterpret_cast<uint4 *>(tile + (c >> 3) * (L::kBlock) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(0, 0, 0, 0);
        }
    ptx::fence_proxy_async_smem();
}

// The terms of drafts that are not finite, for the rows that attend to them: weight
// and value from memory.  o: dims from d0 on of this row's unnormalised sums over m.
__device__ __noinline__ void add_bad(const AttnArgs &A, const AttnPiece &pc, unsigned long long bad, int64_t qrow, float m,
                                     int d0, int dims, float *o) {
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
        for (int d = 0; d < dims; ++d) o[d] = fmaf(p, __bfloat162float(v[d0 + d]), o[d]);
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
    uint32_t used = 0, pieces = 0;                          // places used of the values' ring
    uint32_t s_ph = 0, pv_ph = 0;                           // bit of a buffer: parity of the tiles taken, handed on
    bool ok = true;
    AttnWalk walk = attn_walk(A, plan, group);
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
        const int mine = stream_tiles<L>(n, w);
        for (int j = 0; j < mine; ++j) {
            const int buf = j & 1, tile = pc.t0 + stream_tile<L>(j, w), k0 = tile * kTile;
            const bool drafts = k0 + kTile > pc.len;   // the tile holds drafted tokens, or ends the row
            const uint32_t s_addr = lane_addr + L::col_s(w, buf);
            ok = ok && wait(bar(ms->s_full[2 * w + buf]), (s_ph >> buf) & 1u, &ms->abort);
            s_ph ^= 1u << buf;
            ptx::tc_fence_after_sync();
            if (ok && warp_on) {
                uint32_t s[kTile];
                ptx::tmem_ld32_bits(s_addr, s);
                ptx::tmem_ld32_bits(s_addr + 32, s + 32);
                landed(s);
                if (drafts) {
                    const uint64_t bits = visible_bits(k0, pc.len, mask);
#pragma unroll
                    for (int x = 0; x < kTile; ++x)
                        if (!((uint32_t)(bits >> (x & 32)) >> (x & 31) & 1u)) s[x] = 0xff800000u;
                }
                // eight chains of three-input maxima: one chain's latency would be the whole row's
                float tops[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const auto f = [&](int y) { return __uint_as_float(s[x + 8 * y]); };
                    tops[x] = max3(max3(max3(f(0), f(1), f(2)), f(3), f(4)), f(5), fmaxf(f(6), f(7)));
                }
                const float top = c * max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]),
                                           fmaxf(tops[6], tops[7]));
                const bool move = top > m + kGrow;
                if (__any_sync(0xffffffffu, move)) {
                    const float to = move ? top : m;
                    const float al = m == -INFINITY ? 0.0f : ex2(m - to);
                    l *= al;
                    m = to;
                    if (j > 0) {   // O holds the sums up to the stream's tile before this one
                        ok = wait(bar(ms->pv_done[2 * w + (buf ^ 1)]), ((pv_ph >> (buf ^ 1)) & 1u) ^ 1u, &ms->abort);
                        if (ok) {
                            ptx::tc_fence_after_sync();
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                uint32_t u[32];
                                ptx::tmem_ld32_bits(lane_addr + L::col_o(w) + x, u);
                                landed(u);
#pragma unroll
                                for (int y = 0; y < 32; ++y) u[y] = __float_as_uint(__uint_as_float(u[y]) * al);
                                ptx::tmem_st16_bits(lane_addr + L::col_o(w) + x, u);
                                ptx::tmem_st16_bits(lane_addr + L::col_o(w) + x + 16, u + 16);
                            }
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.0f : -m;
                const uint64_t c2 = pair(c, c), off2 = pair(off, off);
                uint64_t sum[4] = {0, 0, 0, 0};   // pairs of zeros
#pragma unroll
                for (int x = 0; x < kTile; x += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(s[x + 2 * y]), __uint_as_float(s[x + 2 * y + 1])), c2, off2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[y & 3] = add2(sum[y & 3], pair(a, b));
                        p[y] = pack_bf16(a, b);
                    }
                    ptx::tmem_st16_bits(s_addr + x / 2, p);
                }
                float s0, s1;
                unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                l += s0 + s1;
                ptx::tmem_st_wait();
            }
            if (drafts && (!L::kShare || w == 0)) {
                const uint32_t pos = used + j / L::kUnit, st = L::first(L::ring_of(w)) + pos % L::NV;
                ok = ok && wait(bar(ms->full[st]), (pos / L::NV) & 1u, &ms->abort);
                clean_values<D, NQ>(sm + L::kOffKV + st * L::kStage + (j & (L::kUnit - 1)) * L::kBlocks * L::kBlock, k0,
                                    pc.len, kv, tid, &ms->bad[pieces % 3]);
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if ((tid & 31) == 0) ptx::mbar_arrive(bar(ms->p_full[2 * w + buf]));
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
            constexpr int kDims = L::kTurns ? D / 2 : D;   // of D, the head's dims filled up to 64, 128 or 256
            const int d_begin = L::kTurns ? w * kDims : 0;
            const int64_t part = (int64_t)blockIdx.x * 2 + pc.side;
            const bool whole = pc.whole();
            // a piece to be joined is kept as it is (a lane with a draft that is not finite takes the long way)
            const bool kept = !L::kTurns && !whole && !__any_sync(0xffffffffu, bad != 0);
            if (kept) {
#pragma unroll 1
                for (int x = 0; x < kDims && x < A.C.D; x += 64) {
                    uint32_t u[64];
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(w) + x, u);
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(w) + x + 32, u + 32);
                    landed(u);
                    float4 *po = A.part_o + (part * (A.C.D / 4) + x / 4) * A.MT + my_row;
#pragma unroll
                    for (int y = 0; y < 64; y += 4)
                        if (on && x + y < A.C.D)
                            po[(int64_t)(y / 4) * A.MT] =
                                make_float4(__uint_as_float(u[y]), __uint_as_float(u[y + 1]), __uint_as_float(u[y + 2]),
                                            __uint_as_float(u[y + 3]));
                }
            }
            constexpr int kBatch = 32;   // a short body: it is fetched anew for every piece
#pragma unroll 1
            for (int x = kept ? kDims : 0; x < kDims && d_begin + x < A.C.D; x += kBatch) {
                const int d0 = d_begin + x, dims = min(kBatch, A.C.D - d0);
                uint32_t u[kBatch], v[L::kTurns ? kBatch : 1];
#pragma unroll
                for (int y = 0; y < kBatch; y += 32) {
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(L::kTurns ? 0 : w) + d0 + y, u + y);
                    if (L::kTurns) ptx::tmem_ld32_bits(lane_addr + L::col_o(1) + d0 + y, v + (L::kTurns ? y : 0));
                }
                landed(u);
                if (L::kTurns) landed(v);
                float f[kBatch];
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {   // a stream that saw nothing may hold anything
                    if (L::kTurns)
                        f[y] = (w0 != 0.0f ? __uint_as_float(u[y]) * w0 : 0.0f) +
                               (w1 != 0.0f ? __uint_as_float(v[L::kTurns ? y : 0]) * w1 : 0.0f);
                    else
                        f[y] = l != 0.0f ? __uint_as_float(u[y]) : 0.0f;
                }
                if (on) {
                    if (bad) {   // rare: a copy of its own, so that f stays in registers
                        float g[kBatch];
#pragma unroll
                        for (int y = 0; y < kBatch; ++y) g[y] = f[y];
                        add_bad(A, pc, bad, row, m, d0, dims, g);
#pragma unroll
                        for (int y = 0; y < kBatch; ++y) f[y] = g[y];
                    }
                    if (whole) {
                        uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(A.out) + row * A.C.D + d0);
#pragma unroll
                        for (int y = 0; y < kBatch; y += 8)
                            if (y < dims)
                                out[y / 8] = make_uint4(pack_bf16(f[y] * inv, f[y + 1] * inv),
                                                        pack_bf16(f[y + 2] * inv, f[y + 3] * inv),
                                                        pack_bf16(f[y + 4] * inv, f[y + 5] * inv),
                                                        pack_bf16(f[y + 6] * inv, f[y + 7] * inv));
                    } else {
                        float4 *po = A.part_o + (part * (A.C.D / 4) + d0 / 4) * A.MT + my_row;
#pragma unroll
                        for (int y = 0; y < kBatch; y += 4)
                            if (y < dims) po[(int64_t)(y / 4) * A.MT] = make_float4(f[y], f[y + 1], f[y + 2], f[y + 3]);
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
        used += (mine + L::kUnit - 1) / L::kUnit;
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
    const int tid = threadIdx.x, warp = tid >> 5;
    const int group = blockIdx.x / A.NQT, qt = blockIdx.x - group * A.NQT;
    uint32_t have;
    asm("mov.u32 %0, %dynamic_smem_size;" : "=r"(have));
    if (pad + L::kOffMisc + sizeof(Misc) > have) {   // the segment does not start where it always has
        grid_dep_wait();
        if (tid == 0) {
            atomicOr(A.C.status, GDN_SPEC_ST_TIMEOUT);
            if (qt == 0) attn_note(A, group, false, AttnPiece(), 1);   // the join finds an empty chunk
        }
        return;
    }
    if (tid == 0) {
        const auto init = [](uint64_t &b, uint32_t n) { ptx::mbar_init(ptx::smem_addr(&b), n); };
        for (int i = 0; i < L::NST; ++i) {
            init(ms->full[i], 1);
            init(ms->empty[i], i < L::NK ? NQ : 1);   // warps that use the stage
        }
        for (int i = 0; i < 2; ++i) {
            init(ms->q_full[i], 1);
            init(ms->q_empty[i], NQ);
        }
        for (int i = 0; i < 4; ++i) {
            init(ms->s_full[i], 1);
            init(ms->p_full[i], 4);
            init(ms->pv_done[i], 1);
        }
        init(ms->o_full, L::kTurns ? 2 : 1);
        init(ms->o_empty, L::NWG * 4);
        for (int i = 0; i < 3; ++i) init(ms->drain[i], 1);
        ms->bad[0] = ms->bad[1] = ms->bad[2] = 0;
        ms->abort = 0;
        ptx::mbar_init_fence();
        ptx::prefetch_tmap(&mq);
        ptx::prefetch_tmap(&mk);
        ptx::prefetch_tmap(&mv);
    }
    if (warp == 0) ptx::tmem_alloc(ptx::smem_addr(&ms->tmem), kTmemCols);
    grid_dep_wait();   // nothing in global memory was touched so far
    const AttnPlan plan = attn_plan<L::kThreads>(A, group, blockIdx.x == 0, ms->scratch);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;

    if (warp < L::NWG * 4) {
        // while the first tile is on its way
        attn_dead_rows<__nv_bfloat16>(A, blockIdx.x, gridDim.x, tid, L::NWG * 128);
        soften<D, NQ>(A, ms, sm, tmem, plan, group, qt, tid);
    } else {
        const int role = warp - L::NWG * 4;
        if (role == 0) produce<D, NQ>(A, &mq, &mk, &mv, ms, base, plan, group, qt);
        else if (role <= NQ) multiply_scores<D, NQ>(A, ms, base, tmem, plan, group, qt, role - 1);
        else if (role <= NQ + (L::kTurns ? 2 : 1)) multiply_sums<D, NQ>(A, ms, base, tmem, plan, group, qt, role - NQ - 1);
        __syncwarp();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0 && ms->abort) atomicOr(A.C.status, GDN_SPEC_ST_TIMEOUT);
    grid_dep_launch();
}

// ------------------------------------------------------------------ host

template <int D, int NQ>
cudaError_t run(const AttnArgs &A, cudaStream_t st) {
    using L = Lay<D, NQ>;
    static_assert(L::kOffMisc + sizeof(Misc) <= kSmemMax && kTile == 1 << 6, "shared memory, tile");
    // room to reach a 1024-byte boundary (the dynamic segment starts on one: there is no static one)
    constexpr size_t need = L::kOffMisc + sizeof(Misc) + 1024;
    constexpr size_t smem = need < (size_t)kSmemMax ? need : (size_t)kSmemMax;
    static KernelSetup setup;
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)tree_attn_tc_kernel<D, NQ>, smem, &sms);
    if (e != cudaSuccess) return e;
    const cuuint64_t rows = (cuuint64_t)A.C.n_layers * A.C.num_pages * A.C.HKV * A.C.P;
    // Keys and values as (64 dims, token rows, blocks of 64 dims) where a box can hold all of a tile's blocks (they land
    // one after another), else as (dims, token rows, 1) with a box for each block; dims past the head's are filled
    // with zeros.
    const cuuint64_t dims = A.C.D;
    const cuuint64_t kv_dims[3] = {A.whole ? 64 : dims, rows, A.whole ? dims / 64 : 1}, kv_stride[2] = {dims, 64};
    const cuuint32_t kv_box[3] = {64, (cuuint32_t)(A.C.P < kTile ? A.C.P : kTile), A.whole ? (cuuint32_t)(dims / 64) : 1u};
    const int tokens_q = A.MT / NQ / A.G;
    const cuuint64_t q_dims[3] = {dims, (cuuint64_t)A.HQ, (cuuint64_t)A.B * A.T};
    const cuuint64_t q_stride[2] = {dims, (cuuint64_t)A.HQ * dims};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)A.G, (cuuint32_t)(tokens_q < A.T ? tokens_q : A.T)};
    CUtensorMap mq, mk, mv;
    if (!bf16_map(&mk, A.C.k, 3, kv_dims, kv_stride, kv_box) || !bf16_map(&mv, A.C.v, 3, kv_dims, kv_stride, kv_box) ||
        !bf16_map(&mq, A.q, 3, q_dims, q_stride, q_box))
        return cudaErrorInvalidValue;
    return launch_dependent(tree_attn_tc_kernel<D, NQ>, dim3(A.groups * A.NQT), dim3(L::kThreads), smem, st, mq, mk, mv, A);
}

}  // namespace tat

bool tree_attn_tc_supported(const KvArgs &C, int G, bool bf16) {
    return bf16 && G <= tat::kRows && (int64_t)C.n_layers * C.num_pages * C.HKV * C.P <= INT32_MAX;
}

// The cut of the work: a query tile holds whole tokens, as many as fit in 128 rows;
// windows beyond one tile take two side by side where TMEM holds both (D <= 128).
void tree_attn_tc_cut(AttnArgs *A, int sms) {
    const int R = A->T * A->G, tile = tat::kRows / A->G * A->G;
    const int nq = A->C.D <= 128 && R > tile ? 2 : 1;
    A->whole = A->C.P >= tat::kTile && A->C.D % 64 == 0 && A->C.D != 192;
    A->TN = tat::kTile;
    A->MT = nq * tile;
    A->NQT = (R + A->MT - 1) / A->MT;
    const int groups = sms / A->NQT;
    A->groups = groups < 1 ? 1 : groups;
    A->min_chunk = 1;
    // what an item costs besides its tiles, in tiles: of 0, 2, 4, 6 and 8 the best over a hundred shapes (6 against 0:
    // 32.6 and 35.6 us in the geometric mean with heads of 128; 4 against 0: 69.1 and 71.3 us with heads of 256)
    A->gap = A->C.D > 128 ? 4 : 6;
}

cudaError_t launch_tree_attn_tc(const AttnArgs &A, cudaStream_t st) {
    const bool two = A.MT > tat::kRows;
    cudaError_t e;
    if (A.C.D <= 64) e = two ? tat::run<64, 2>(A, st) : tat::run<64, 1>(A, st);
    else if (A.C.D <= 128) e = two ? tat::run<128, 2>(A, st) : tat::run<128, 1>(A, st);
    else e = tat::run<256, 1>(A, st);
    return e != cudaSuccess ? e : launch_attn_join(A, true, st);
}

}  // namespace gdnspec
