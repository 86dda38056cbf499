// prompt_attn_tc.cu -- attention of packed prompts over the paged cache on the tensor
// cores (bf16; heads of other than 64, 128 or 256 dims are filled up with zeros to the
// next of them in shared memory).
//
// A block works through the pieces of its chunk (prompt_common.cuh) in tiles of 128 keys:
//   S = Q K^T     tcgen05.mma kind::f16, 128 query rows x 128 keys, fp32 in TMEM
//   P = 2^(S scale log2 e - m), rounded to bf16, back into TMEM over S
//   O += P V      tcgen05.mma kind::f16, P from TMEM, V as it lies in its pages
//                 (token rows of 64-element runs: the MN-major operand), fp32 in TMEM
// D <= 128: two streams of 128 query rows, a warpgroup for the softmax of each, share every
// key and value tile; while one's scores are softened, the other's products run.
// D = 256: one stream, whose O takes half of TMEM, with its scores in two buffers, so that
// the next tile's scores are formed while a softmax runs.
//
// Warps of their own copy the pages' rows by TMA into rings of stages (and walk and describe
// the pieces to the others), issue the products, and look through the values
// (below).  With two streams a warp issues all products of one: they run in order, so a
// stream's next scores are issued right behind the sums that read the probabilities in the same
// columns, without a wait between them.
//
// What bounds it is a stream's round: softmax, 950 cycles at best (MUFU: 512 for the
// exponentials), sums and scores, 1024, and four hand-overs through barriers.  Two streams
// fill the tensor core to 72% that way (4 x 1024 tokens behind 19751 to 30000, 16 heads on 2 of 128: 525 to 545 us,
// 1.56 to 1.62 PFLOP/s; 8192 tokens, 32 on 8 of 128: 371 to 394 us, 1.40 to 1.48; heads of 64, where a round
// multiplies half as much: the first case in 447 us, 0.95 PFLOP/s).  What led there, first case: 770 us; scores in quarters
// and walkers out of line, so that the loops stay in the instruction cache (a kernel of 170 KB
// of code waited for instructions a third of the softmax's time): 600; pieces described once: 554;
// probabilities in one pass against the maximum so far: 525.  Not faster: waiting by looking
// at a barrier in a loop (13% slower: it takes the softmax's issue slots); one warp for both
// streams' products (600 us as it stood then); both streams issuing at will (607); for D = 256 pairs of
// blocks that share tiles by multicast.  D = 256: 16384 + 10308 tokens, 16 heads on 2: 1960 to
// 2170 us over several GB300s, 1.41 to 1.57 PFLOP/s.
//
// The running maximum is only moved when a row's maximum has grown by more than 2^8 over
// it, an idea published for attention kernels of this generation: until then the
// probabilities are taken against the old one, which is exact (they and their sum stay below 2^8
// times as large, far inside fp32 and bf16's range), and O is not read and rescaled.  P is
// rounded to bf16 because it is an operand of the second product; m, l and O are fp32, and
// l is the sum of the values before that rounding, so that lse keeps fp32's accuracy (out is
// off by 0.0020 to 0.0023 of itself against 64 bits, its own rounding alone is 0.0017).
//
// Rows of a tile past the last token hold whatever the page or the buffer held, and a token
// behind the one that asks may hold anything; 0 times NaN is not 0.  So in the tiles
// that not every row of the block sees whole, a warp looks for value rows that are
// not finite, before the products get the tile, and zeroes them; the terms of those that
// some rows see are added to these rows at the end.
//
// Every wait is bounded.  One that runs out raises the block's abort flag, on which all
// roles leave their loops; the producers then wait for the copies they have in flight and
// the MMA warps for their MMAs, TMEM is freed, and the status word gets TIMEOUT.
#include <cstddef>
#include <type_traits>

#include "attn_tc.cuh"
#include "launch_setup.cuh"
#include "prompt_common.cuh"

namespace gdnspec {
namespace pat {

using tat::ex2;
using tat::landed;
using tat::max3;
using tat::pack_bf16;
using tat::pair;
using tat::uniform;
using tat::unpair;
using tat::wait;

constexpr int kRows = 128;               // query rows of an MMA
constexpr int kLogTile = 7, kTile = 1 << kLogTile;   // keys of a tile
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemMax = 232448;
constexpr int kMaxStages = 10;
constexpr int kNotes = 4;                // pieces whose rows that are not finite are kept
constexpr int kPieces = 4;               // pieces that are described at a time

template <int D>
struct Lay {
    static constexpr int NS = D == 256 ? 1 : 2;                // streams
    static constexpr int kProducers = NS == 1 ? 2 : 1;         // warps that copy
    static constexpr int kThreads = NS * 128 + 96 + kProducers * 32;   // softmax warpgroups; producers, two for the MMAs, cleaner
    static constexpr int kParts = D == 256 ? 2 : 1;            // stages of a tile: keys in halves of the dims, values of the tokens
    static constexpr uint32_t kKBlocks = D / 64 / kParts;      // 64-dim blocks of a stage of keys
    static constexpr uint32_t kVBlocks = D / 64;               // of values
    static constexpr int kVRows = kTile / kParts;              // tokens of a stage of values
    static constexpr uint32_t kKBlock = kTile * 128, kVBlock = kVRows * 128;
    static constexpr uint32_t kStage = kTile * D * 2 / kParts;
    static constexpr uint32_t kQTile = kRows * D * 2;
    // Stages stand in two rings, of keys and of values, so that a stage's barriers are met by the same warps in every phase.
    static constexpr int NK = D == 64 ? 5 : 2, NV = D == 64 ? 5 : 3, NST = NK + NV;
    static constexpr uint32_t kOffKV = NS * kQTile;
    static constexpr uint32_t kOffMisc = kOffKV + NST * kStage;
    // TMEM columns: two buffers of S (one for each of two streams), then O
    __host__ __device__ static constexpr uint32_t col_s(int x) { return x * kTile; }
    __host__ __device__ static constexpr uint32_t col_o(int s) { return 256 + s * 128; }
};

// A piece as its readers need it.  The producer walks and describes the pieces in shared memory, a few ahead: walkers of
// all warps' own would cost each of them some thousand cycles a piece.
struct __align__(16) PieceInfo {
    int slot, len, cnt, first;            // the row: its slot, committed tokens, tokens, and the first of them
    int h, part, q0, keys;                // as in PromptItem
    int tiles, t0, n[2];                  // tiles of the item, the piece's first, tiles that each stream takes
    int units, all, whole, chunk;         // tiles of the piece (0: there is none), keys that all its rows see, whether it is the item, the chunk
};

// Value rows of a piece that are not finite, from its first key that not all rows see on.
struct Note {
    int piece;                            // the piece's number; another one's: there are none
    unsigned long long rows[4];
};

// Shared memory behind the tiles.
struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages], clean[kMaxStages];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2], pv_done[2], turn[2], drain[2];
    PieceInfo pieces[kPieces];
    Note notes[kNotes];
    int done[8];                          // pieces that a warp of the softmax is done with
    PromptScratch scratch;
    uint32_t tmem;
    int abort;
};

// The barriers' addresses.
struct Bars {
    uint32_t misc;
    __device__ __forceinline__ uint32_t at(size_t offset, uint32_t i) const { return misc + (uint32_t)offset + 8u * i; }
    __device__ __forceinline__ uint32_t full(uint32_t i) const { return at(offsetof(Misc, full), i); }
    __device__ __forceinline__ uint32_t empty(uint32_t i) const { return at(offsetof(Misc, empty), i); }
    __device__ __forceinline__ uint32_t clean(uint32_t i) const { return at(offsetof(Misc, clean), i); }
    __device__ __forceinline__ uint32_t piece_full(uint32_t i) const { return at(offsetof(Misc, piece_full), i); }
    __device__ __forceinline__ uint32_t piece_empty(uint32_t i) const { return at(offsetof(Misc, piece_empty), i); }
    __device__ __forceinline__ uint32_t q_full(uint32_t i) const { return at(offsetof(Misc, q_full), i); }
    __device__ __forceinline__ uint32_t q_empty(uint32_t i) const { return at(offsetof(Misc, q_empty), i); }
    __device__ __forceinline__ uint32_t s_full(uint32_t i) const { return at(offsetof(Misc, s_full), i); }
    __device__ __forceinline__ uint32_t p_full(uint32_t i) const { return at(offsetof(Misc, p_full), i); }
    __device__ __forceinline__ uint32_t o_full(uint32_t i) const { return at(offsetof(Misc, o_full), i); }
    __device__ __forceinline__ uint32_t o_empty(uint32_t i) const { return at(offsetof(Misc, o_empty), i); }
    __device__ __forceinline__ uint32_t pv_done(uint32_t i) const { return at(offsetof(Misc, pv_done), i); }
    __device__ __forceinline__ uint32_t turn(uint32_t i) const { return at(offsetof(Misc, turn), i); }
    __device__ __forceinline__ uint32_t drain(uint32_t i) const { return at(offsetof(Misc, drain), i); }
};

// The next piece's description from the ring, for a warp that goes through the pieces; false: there is none, or the
// wait ran out (*ok).
struct PieceReader {
    uint32_t at = 0, ph = 0;
    __device__ __forceinline__ bool next(Misc *ms, const Bars &bars, PieceInfo *info, bool *ok) {
        *ok = wait(bars.piece_full(at), ph, &ms->abort);
        if (!*ok) return false;
        *info = ms->pieces[at];
        __syncwarp();
        if (ptx::elect_one()) ptx::mbar_arrive(bars.piece_empty(at));
        if (++at == kPieces) {
            at = 0;
            ph ^= 1u;
        }
        return info->units > 0;
    }
};

// Place in the ring of keys or of values: the stage and its phase.
template <int D, bool KEYS>
struct Ring {
    uint32_t at = KEYS ? 0 : Lay<D>::NK, ph = 0;
    __device__ __forceinline__ void step() {
        if (++at == (KEYS ? Lay<D>::NK : Lay<D>::NST)) {
            at = KEYS ? 0 : Lay<D>::NK;
            ph ^= 1u;
        }
    }
};

// ------------------------------------------------------------------ producer warps

// One lane issues: a copy's operands are uniform registers.  The lanes look up the pages of a tile's boxes side by side.
// With two streams one warp copies keys and values of each tile in turn; with one, whose rings hold little more than a
// tile, keys and values have a warp each, so that neither waits for the other's stage (4 x 1024 tokens behind 19751 to 30000, 16
// heads on 2 of 256: 1266 us with one warp, 1227 with two).  The keys' warp walks, describes the pieces and
// copies the queries.
template <int D, bool KEYS, bool VALUES>
__device__ __forceinline__ void produce(const PromptArgs &A, const CUtensorMap *mq, const CUtensorMap *mk,
                                        const CUtensorMap *mv, Misc *ms, uint32_t base, const PromptPlan &plan) {
    using L = Lay<D>;
    const int lane = threadIdx.x & 31;
    const int log_br = min(A.C.logP, 7), BR = 1 << log_br;     // tokens of a box: within a page and within a tile
    const int tq = A.tokens / L::NS;
    const uint32_t q_bytes = 128u * A.GS * min(tq, A.N);       // one 64-dim block of one query tile
    Ring<D, true> k_ring;
    Ring<D, false> v_ring;
    uint32_t issued[2] = {0, 0};                               // stages of values, of keys
    uint32_t q_issued = 0, q_any = 0;                          // bit of a stream: parity of its query tiles, whether there was one
    bool ok = true;
    int wave = 0;
    PromptWalk walk;
    if (KEYS) {
        walk = PromptWalk(A, plan, 0);
        if (ptx::elect_one()) prompt_note(A, walk, plan.chunk, 0);
        __syncwarp();
    }
    PromptPiece pc;
    PieceReader reader;                                        // (of the values' warp)
    uint32_t at = 0, ph = 1;                                   // place in the ring of pieces
    // the piece pc's description; at the end (!any) that there is none
    const auto describe = [&](bool any, PieceInfo *info) {
        info->units = 0;
        if (any) {
            const PromptItem &it = pc.it;
            info->slot = it.slot, info->len = it.len, info->cnt = it.cnt, info->first = it.first;
            info->h = it.h, info->part = it.part, info->q0 = it.q0, info->keys = it.keys;
            info->tiles = it.tiles, info->t0 = pc.t0, info->n[1] = 0;
#pragma unroll
            for (int s = 0; s < L::NS; ++s) {
                const int first = it.q0 + s * tq;              // the stream's first token
                const int keys = first < it.cnt ? it.len + min(it.cnt, first + tq) : 0;
                info->n[s] = max(0, min(pc.t1, (keys + kTile - 1) >> kLogTile) - pc.t0);
                info->units = max(info->units, info->n[s]);
            }
            info->all = it.len + it.q0 + 1;
            info->whole = pc.whole();
            info->chunk = wave * A.groups + blockIdx.x;
        }
        if (!wait(ptx::smem_addr(&ms->piece_empty[at]), ph, &ms->abort)) return false;
        if (ptx::elect_one()) {
            ms->pieces[at] = *info;
            ptx::mbar_arrive(ptx::smem_addr(&ms->piece_full[at]));
        }
        __syncwarp();
        if (++at == kPieces) {
            at = 0;
            ph ^= 1u;
        }
        return true;
    };
    // one stage of keys or values of the tile at `tok`, whose boxes' pool rows are `row`
    const auto stage = [&](auto &ring, auto keys_c, int part, int row, int boxes) {
        constexpr bool keys = decltype(keys_c)::value;
        if (!wait(ptx::smem_addr(&ms->empty[ring.at]), ring.ph ^ 1u, &ms->abort)) return false;
        const uint32_t bar = uniform(ptx::smem_addr(&ms->full[ring.at])), dst = uniform(base + L::kOffKV + ring.at * L::kStage);
        const CUtensorMap *map = keys ? mk : mv;
        const int rows_here = keys ? kTile : L::kVRows;        // tokens of the stage
        const int box = min(BR, rows_here);                    // of a copy
        const int first = keys ? 0 : part * L::kVRows;         // token of the tile where the stage starts
        constexpr int blocks = keys ? L::kKBlocks : L::kVBlocks;
        const int blk0 = keys ? part * L::kKBlocks : 0;
        const uint32_t block = keys ? L::kKBlock : L::kVBlock;
        // boxes of `box` tokens that lie before the end
        const int n = max(0, min((boxes * BR - first) >> (31 - __clz(box)), rows_here >> (31 - __clz(box))));
        const bool whole = keys ? A.k_whole : A.v_whole;
        int mine = 0;   // pool row of copy `lane` of this stage
        {
            const int tok = first + lane * box;                // of the tile
            mine = __shfl_sync(0xffffffffu, row, min(31, tok >> log_br)) + (tok & (BR - 1));
        }
        if (whole) {
            const int r = __shfl_sync(0xffffffffu, mine, 0);
            if (ptx::elect_one()) {
                ptx::mbar_expect_tx(bar, n ? L::kStage : 0);
                if (n) ptx::tma_load_3d(dst, map, bar, 0, r, blk0);
            }
        } else {
            int rows[kTile / 16];
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c) rows[c] = __shfl_sync(0xffffffffu, mine, c);
            if (ptx::elect_one()) {
                ptx::mbar_expect_tx(bar, (uint32_t)box * 128u * blocks * n);
#pragma unroll
                for (int c = 0; c < kTile / 16; ++c) {
                    if (c >= n) break;
#pragma unroll
                    for (int b = 0; b < blocks; ++b)
                        ptx::tma_load_3d(dst + b * block + c * box * 128u, map, bar, (blk0 + b) * 64, rows[c], 0);
                }
            }
        }
        __syncwarp();
        ++issued[keys];
        ring.step();
        return true;
    };
    while (ok) {
        PieceInfo sp;
        bool any;
        if (KEYS) {
            any = walk.next(A, plan, &pc);
            while (!any && wave + 1 < A.waves) {   // the block's next chunk
                walk = PromptWalk(A, plan, ++wave);
                if (ptx::elect_one()) prompt_note(A, walk, plan.chunk, wave);
                __syncwarp();
                any = walk.next(A, plan, &pc);
            }
            ok = describe(any, &sp);
        } else {
            any = reader.next(ms, Bars{ptx::smem_addr(ms)}, &sp, &ok);
        }
        if (!ok || !any) break;
        const int kv = min(sp.keys, (sp.t0 + sp.units) * kTile);
        const int32_t *table = A.C.page_table + (int64_t)sp.slot * A.C.max_pages;
        // the page of box `lane` of tile u: looked up two tiles before it is used
        const auto page_of = [&](int u) {
            const int tok = (sp.t0 + u) * kTile + lane * BR;
            return u < sp.units && lane * BR < kTile && tok < kv ? table[tok >> A.C.logP] : 0;
        };
        const auto row_of = [&](int u, int page) {
            const int tok = (sp.t0 + u) * kTile + lane * BR;
            if (lane * BR < kTile && tok < kv && (page < 0 || page >= A.C.num_pages)) {
                atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
                page = 0;
            }
            return ((A.layer * A.C.num_pages + page) * A.C.HKV + sp.h) * A.C.P + (tok & (A.C.P - 1));
        };
        int page = page_of(0), next = page_of(1);
#pragma unroll 1
        for (int u = 0; ok && u < sp.units; ++u) {
            const int row = row_of(u, page), boxes = (min(kTile, kv - (sp.t0 + u) * kTile) + BR - 1) >> log_br;
            page = next;
            next = page_of(u + 2);
            if (KEYS)
#pragma unroll 1
                for (int p = 0; ok && p < L::kParts; ++p) ok = stage(k_ring, std::true_type(), p, row, boxes);
            if (KEYS && u == 0) {   // the query tiles, behind the first keys
#pragma unroll 1
                for (int s = 0; s < L::NS; ++s) {
                    if (!ok || (s ? sp.n[1] : sp.n[0]) == 0) continue;
                    ok = wait(ptx::smem_addr(&ms->q_empty[s]), ((q_issued >> s) & 1u) ^ 1u, &ms->abort);
                    if (!ok) break;
                    const uint32_t bar = uniform(ptx::smem_addr(&ms->q_full[s])), dst = uniform(base + s * L::kQTile);
                    if (ptx::elect_one()) {
                        ptx::mbar_expect_tx(bar, q_bytes * L::kVBlocks);
#pragma unroll
                        for (int blk = 0; blk < (int)L::kVBlocks; ++blk)
                            ptx::tma_load_3d(dst + blk * (kRows * 128u), mq, bar, blk * 64, sp.h * A.G + sp.part * A.GS,
                                             sp.first + sp.q0 + s * tq);
                    }
                    __syncwarp();
                    q_issued ^= 1u << s;
                    q_any |= 1u << s;
                }
            }
            if (VALUES)
#pragma unroll 1
                for (int p = 0; ok && p < L::kParts; ++p) ok = stage(v_ring, std::false_type(), p, row, boxes);
        }
    }
    if (KEYS)   // (a walk that was broken off leaves its later chunks to be found empty)
        for (++wave; wave < A.waves; ++wave) {
            if (ptx::elect_one()) prompt_note(A, PromptWalk(), 1, wave);
            __syncwarp();
        }
    if (!ok) {   // copies in flight land before the block's shared memory goes away
        for (uint32_t p = issued[1] > L::NK ? issued[1] - L::NK : 0; p < issued[1]; ++p)
            ptx::mbar_wait(ptx::smem_addr(&ms->full[p % L::NK]), (p / L::NK) & 1u);
        for (uint32_t p = issued[0] > L::NV ? issued[0] - L::NV : 0; p < issued[0]; ++p)
            ptx::mbar_wait(ptx::smem_addr(&ms->full[L::NK + p % L::NV]), (p / L::NV) & 1u);
#pragma unroll
        for (int s = 0; s < L::NS; ++s)
            if ((q_any >> s) & 1u) ptx::mbar_wait(ptx::smem_addr(&ms->q_full[s]), ((q_issued >> s) & 1u) ^ 1u);
    }
}

// ------------------------------------------------------------------ MMA warps

// A place in the sequence of tiles, piece after piece: tile u of a piece's `units`, of which stream s takes n.
struct Cursor {
    int u = 0, units = 0, n = 0;
    bool live = false;
    // Opens the next piece.
    __device__ __forceinline__ void open(Misc *ms, const Bars &bars, PieceReader &reader, int s, bool *ok) {
        PieceInfo info;
        live = reader.next(ms, bars, &info, ok);
        u = 0;
        units = info.units;
        n = s ? info.n[1] : info.n[0];
    }
};

// What an MMA needs is made uniform before the waits that it hangs on, so that only the issue is behind them; one
// lane issues, and commits to the barriers that follow.  In the elected lane only:

// Scores of one stage of keys (b) with the query tile's dims that go with them (a) into d; add: onto what d holds.
template <int D>
__device__ __forceinline__ void scores_mma(uint32_t d, uint64_t a, uint64_t b, bool add) {
    using L = Lay<D>;
    constexpr uint32_t idesc = ptx::idesc_bf16(kRows, kTile);
#pragma unroll
    for (int ks = 0; ks < (int)L::kKBlocks * 4; ++ks)   // descriptors count in 16 bytes
        ptx::mma_bf16(d, a + ((ks >> 2) * (kRows * 128u) + (ks & 3) * 32u) / 16,
                      b + ((ks >> 2) * L::kKBlock + (ks & 3) * 32u) / 16, idesc, add || ks != 0);
}

// Sums over one stage of values (b) with its probabilities (p) into d.
template <int D>
__device__ __forceinline__ void sums_mma(uint32_t d, uint32_t p, uint64_t b, uint32_t add) {
    using L = Lay<D>;
    constexpr uint32_t idesc = ptx::idesc_bf16(kRows, D) | ptx::kIdescBMn;
#pragma unroll
    for (int ks = 0; ks < L::kVRows / 16; ++ks)
        ptx::mma_bf16_tmem_a(d, p + ks * 8, b + ks * 2048u / 16, idesc, ks != 0 ? 1u : add);
}

template <int D> __device__ __forceinline__ uint64_t keys_desc(uint32_t base, uint32_t stage) {
    return ptx::smem_desc_sw128(uniform(base + Lay<D>::kOffKV + stage * Lay<D>::kStage));
}
template <int D> __device__ __forceinline__ uint64_t values_desc(uint32_t base, uint32_t stage) {
    return ptx::smem_desc_sw128_mn(uniform(base + Lay<D>::kOffKV + stage * Lay<D>::kStage), Lay<D>::kVBlock);
}

// When a warp gives up, none of its MMAs is running when TMEM is freed.
__device__ __forceinline__ void drain(const Bars &bars, int who) {
    tat::commit(bars.drain(who));
    ptx::mbar_wait(bars.drain(who), 0);
}

// Two streams: all products of stream s by one warp, the other's by another, so that what one does between its issues (its
// waits and its bookkeeping take some hundred cycles) is covered by the other's MMAs.  They issue in turns, a tile's
// sums and the next tile's scores at a time: issued side by side both streams' products would end at the same time,
// then both softmaxes would run at the same time, and the tensor core would be idle meanwhile.  A tile that the
// stream takes no part in is released when it has landed.
template <int D>
__device__ __forceinline__ void multiply_stream(const PromptArgs &A, Misc *ms, uint32_t base, uint32_t tmem,
                                                int s) {
    using L = Lay<D>;
    const Bars bars{ptx::smem_addr(ms)};
    Ring<D, true> k_ring;
    Ring<D, false> v_ring;
    uint32_t q_ph = 0, p_ph = 0, o_ph = 1, turn_ph = s ^ 1u;   // the first stream has the first turn
    const uint32_t s_col = uniform(tmem + L::col_s(s)), o_col = uniform(tmem + L::col_o(s));
    const uint64_t a = ptx::smem_desc_sw128(uniform(base + s * L::kQTile));
    const uint32_t s_full = uniform(bars.s_full(s)), q_empty = uniform(bars.q_empty(s)), o_full = uniform(bars.o_full(s)),
                   other = uniform(bars.turn(s ^ 1));
    bool ok = true;
    PieceReader reader;
    Cursor q, p;                   // scores run a tile ahead of sums
    const auto wait_keys = [&] {
        ok = ok && wait(bars.full(k_ring.at), k_ring.ph, &ms->abort, A.wait_limit);
        if (q.u == 0 && q.n > 0) {
            ok = ok && wait(bars.q_full(s), q_ph, &ms->abort, A.wait_limit);
            q_ph ^= 1u;
        }
    };
    // a piece's first scores, out of turn: its queries come when the scores of the piece before are done
    const auto first_scores = [&] {
        const uint64_t b = keys_desc<D>(base, k_ring.at);
        const uint32_t empty = uniform(bars.empty(k_ring.at));
        const bool mine = q.n > 0, last = q.n == 1;
        wait_keys();
        if (!ok) return;
        ptx::tc_fence_after_sync();
        if (ptx::elect_one()) {
            if (mine) {
                scores_mma<D>(s_col, a, b, false);
                ptx::mma_commit(s_full);
                ptx::mma_commit(empty);
                if (last) ptx::mma_commit(q_empty);
            } else {
                ptx::mbar_arrive(empty);
            }
        }
        __syncwarp();
        k_ring.step();
    };
    q.open(ms, bars, reader, s, &ok);
    if (q.live) first_scores();
    p = q;
    while (ok && p.live) {
        const bool sums = p.u < p.n, ends = p.u == p.n - 1;
        const uint32_t add = uniform(p.u != 0);
        const bool same = ++q.u < q.units, scores = same && q.u < q.n, q_ends = q.u == q.n - 1;
        const uint64_t bk = keys_desc<D>(base, k_ring.at), bv = values_desc<D>(base, v_ring.at);
        const uint32_t k_empty = uniform(bars.empty(k_ring.at)), v_empty = uniform(bars.empty(v_ring.at));
        ok = wait(bars.clean(v_ring.at), v_ring.ph, &ms->abort, A.wait_limit);
        if (same) wait_keys();
        if (sums) {
            if (p.u == 0) {
                ok = ok && wait(bars.o_empty(s), o_ph, &ms->abort);
                o_ph ^= 1u;
            }
            ok = ok && wait(bars.p_full(s), p_ph, &ms->abort);
            p_ph ^= 1u;
        }
        ok = ok && wait(bars.turn(s), turn_ph, &ms->abort);
        turn_ph ^= 1u;
        if (!ok) break;
        ptx::tc_fence_after_sync();
        if (ptx::elect_one()) {
            if (sums) {
                sums_mma<D>(o_col, s_col, bv, add);
                ptx::mma_commit(v_empty);
                if (ends) ptx::mma_commit(o_full);
            } else {
                ptx::mbar_arrive(v_empty);
            }
            if (scores) {
                scores_mma<D>(s_col, a, bk, false);
                ptx::mma_commit(s_full);
                ptx::mma_commit(k_empty);
                if (q_ends) ptx::mma_commit(q_empty);
            } else if (same) {
                ptx::mbar_arrive(k_empty);
            }
            ptx::mbar_arrive(other);
        }
        __syncwarp();
        v_ring.step();
        if (same) {
            k_ring.step();
            ++p.u;
        } else {   // both go on to the next piece
            q.open(ms, bars, reader, s, &ok);
            if (q.live) first_scores();
            p = q;
        }
    }
    if (!ok) drain(bars, s);
}

// One stream: its scores by one warp, a tile ahead, its sums by another.  (In turns, as above, they are no faster: 1234 us
// against 1227 for 4 x 1024 tokens behind 19751 to 30000, 16 heads on 2 of 256.)
template <int D>
__device__ __forceinline__ void multiply_scores(const PromptArgs &A, Misc *ms, uint32_t base, uint32_t tmem) {
    using L = Lay<D>;
    const Bars bars{ptx::smem_addr(ms)};
    Ring<D, true> ring;
    uint32_t seq = 0, q_ph = 0;
    const uint32_t q_empty = uniform(bars.q_empty(0));
    bool ok = true;
    PieceReader reader;
    Cursor q;
    for (;; ++seq) {
        if (++q.u >= q.units) {
            q.open(ms, bars, reader, 0, &ok);
            if (!q.live) break;
        }
        const int x = seq & 1;
        const uint32_t d = uniform(tmem + L::col_s(x)), s_full = uniform(bars.s_full(x));
        const bool ends = q.u == q.n - 1;
        if (q.u == 0) {
            ok = wait(bars.q_full(0), q_ph, &ms->abort, A.wait_limit);
            q_ph ^= 1u;
        }
        // the buffer is free once the sums of the tile before the last, which read its probabilities, are done
        if (seq > 1) ok = ok && wait(bars.pv_done(x), ((seq >> 1) & 1u) ^ 1u, &ms->abort);
#pragma unroll
        for (int part = 0; part < L::kParts; ++part) {
            const uint64_t a = ptx::smem_desc_sw128(uniform(base + part * (L::kKBlocks * kRows * 128u)));
            const uint64_t b = keys_desc<D>(base, ring.at);
            const uint32_t empty = uniform(bars.empty(ring.at));
            ok = ok && wait(bars.full(ring.at), ring.ph, &ms->abort, A.wait_limit);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            if (ptx::elect_one()) {
                scores_mma<D>(d, a, b, part != 0);
                if (part == L::kParts - 1) ptx::mma_commit(s_full);
                ptx::mma_commit(empty);
                if (part == L::kParts - 1 && ends) ptx::mma_commit(q_empty);
            }
            __syncwarp();
            ring.step();
        }
        if (!ok) break;
    }
    if (!ok) drain(bars, 0);
}

template <int D>
__device__ __forceinline__ void multiply_sums(const PromptArgs &A, Misc *ms, uint32_t base, uint32_t tmem) {
    using L = Lay<D>;
    const Bars bars{ptx::smem_addr(ms)};
    Ring<D, false> ring;
    uint32_t seq = 0, p_ph = 0, o_ph = 1;   // p_ph: bit of a buffer
    const uint32_t o_col = uniform(tmem + L::col_o(0)), o_full = uniform(bars.o_full(0));
    bool ok = true;
    PieceReader reader;
    Cursor p;
    for (;; ++seq) {
        if (++p.u >= p.units) {
            p.open(ms, bars, reader, 0, &ok);
            if (!p.live) break;
        }
        const int x = seq & 1;
        const uint32_t s_col = uniform(tmem + L::col_s(x)), pv_done = uniform(bars.pv_done(x)), add = uniform(p.u != 0);
        const bool ends = p.u == p.n - 1;
        if (p.u == 0) {
            ok = wait(bars.o_empty(0), o_ph, &ms->abort);
            o_ph ^= 1u;
        }
#pragma unroll
        for (int part = 0; part < L::kParts; ++part) {
            const uint64_t b = values_desc<D>(base, ring.at);
            const uint32_t empty = uniform(bars.empty(ring.at));
            ok = ok && wait(bars.clean(ring.at), ring.ph, &ms->abort, A.wait_limit);
            if (part == 0) ok = ok && wait(bars.p_full(x), (p_ph >> x) & 1u, &ms->abort);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            if (ptx::elect_one()) {
                sums_mma<D>(o_col, s_col + part * (L::kVRows / 2), b, part != 0 ? 1u : add);
                ptx::mma_commit(empty);
                if (part == L::kParts - 1) ptx::mma_commit(pv_done);
                if (part == L::kParts - 1 && ends) ptx::mma_commit(o_full);
            }
            __syncwarp();
            ring.step();
        }
        p_ph ^= 1u << x;
        if (!ok) break;
    }
    if (!ok) drain(bars, 1);
}

// ------------------------------------------------------------------ cleaner

// Eight rows of a stage of values, the first `row` of it and `key` of the piece, of which those in `any` (four bits each) are
// not finite: the ones that not every row sees (keys from `all` on) become zeros, and the piece's own are noted.
template <int D>
__device__ __noinline__ bool remove(Misc *ms, uint8_t *tile, int row, int key, int all, int keys, unsigned any, int piece) {
    using L = Lay<D>;
    const int lane = threadIdx.x & 31;
    Note *const note = &ms->notes[piece % kNotes];
    if (note->piece != piece) {   // the place held an earlier piece's: all are done with it
        const volatile int *done = ms->done;
        for (uint32_t it = 0;; ++it) {   // one answer for all lanes, as in wait()
            if (__all_sync(0xffffffffu, lane >= L::NS * 4 || done[lane] > piece - kNotes)) break;
            if (__any_sync(0xffffffffu, it == tat::kPolls || *(volatile int *)&ms->abort)) {
                ms->abort = 1;
                return false;
            }
            __nanosleep(100);
        }
        __syncwarp();
        // the rows first: a stream that takes fewer tiles than the piece has may be looking at the piece's number
        if (lane < 4) note->rows[lane] = 0;
        __threadfence_block();
        __syncwarp();
        if (lane == 0) *(volatile int *)&note->piece = piece;
        __syncwarp();
    }
#pragma unroll 1
    for (int y = 0; y < 8; ++y) {
        if (key + y < all || !((any >> (4 * y)) & 15u)) continue;
        for (int c = lane; c < (int)L::kVBlocks * 8; c += 32)
            *reinterpret_cast<uint4 *>(tile + (c >> 3) * L::kVBlock + (row + y) * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        if (key + y < keys && lane == 0) note->rows[(key + y - all) >> 6] |= 1ull << ((key + y - all) & 63);
    }
    __syncwarp();
    return true;
}

// Looks at every stage of values: where the tile holds keys that some row does not see, rows that are not finite become
// zeros, and those of the piece's own keys are noted.
template <int D>
__device__ __forceinline__ void clean(const PromptArgs &A, Misc *ms, uint8_t *sm) {
    using L = Lay<D>;
    const int lane = threadIdx.x & 31;
    const Bars bars{ptx::smem_addr(ms)};
    Ring<D, false> ring;
    bool ok = true;
    int piece = 0;
    PieceReader reader;
    PieceInfo sp;
    for (; ok && reader.next(ms, bars, &sp, &ok); ++piece) {
        for (int u = 0; ok && u < sp.units; ++u) {
            const int k0 = (sp.t0 + u) * kTile;
            for (int part = 0; ok && part < L::kParts; ++part) {
                ok = wait(bars.full(ring.at), ring.ph, &ms->abort, A.wait_limit);
                if (ok && k0 + kTile > sp.all) {
                    uint8_t *tile = sm + L::kOffKV + ring.at * L::kStage;
                    const int key0 = k0 + part * L::kVRows;                 // the stage's first key
#pragma unroll 1
                    for (int r = 0; ok && r < L::kVRows; r += 8) {
                        if (key0 + r + 8 <= sp.all) continue;
                        // four lanes a row, each 16 of its bytes at a time; odd rows begin with their second half, so that
                        // two rows' pieces fall in different banks
                        __nv_bfloat162 acc = __float2bfloat162_rn(0.0f);
                        const __nv_bfloat162 zero = acc;
                        const uint8_t *row = tile + (r + (lane >> 2)) * 128;
#pragma unroll
                        for (int b = 0; b < (int)L::kVBlocks; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int c = (lane & 3) + 4 * (h ^ ((lane >> 2) & 1));
                                const uint4 x = *reinterpret_cast<const uint4 *>(row + b * L::kVBlock + c * 16);
                                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j)   // an infinity times zero is NaN too
                                    acc = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]), zero, acc);
                            }
                        const unsigned any = __ballot_sync(0xffffffffu, __hisnan(acc.x) || __hisnan(acc.y));
                        if (any) ok = remove<D>(ms, tile, r, key0 + r, sp.all, sp.keys, any, piece);
                    }
                    ptx::fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bars.clean(ring.at));
                ring.step();
            }
        }
    }
}

// ------------------------------------------------------------------ softmax

// The terms of value rows that are not finite, for a row that sees `own` keys from `all` on: weight and value from memory.
// o: dims from d0 on of the row's unnormalised sums over m.
__device__ __noinline__ void add_removed(const PromptArgs &A, const Misc *ms, int piece, const PieceInfo &it, int all, int own,
                                         int64_t qrow, float m, int d0, int dims, float *o) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(A.q) + qrow * A.C.D;
    __threadfence_block();   // the piece's number was read, its rows are read behind it
    for (int i = 0; i < own; ++i) {
        const Note &note = ms->notes[piece % kNotes];
        const bool there = note.piece == piece && ((note.rows[i >> 6] >> (i & 63)) & 1);
        if (!there) continue;
        const int64_t row = kv_token_row(A.C, it.slot, all + i);
        if (row < 0) continue;
        const int64_t e = kv_elem(A.C, A.layer, it.h, row);
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(A.C.k) + e, *v = static_cast<const __nv_bfloat16 *>(A.C.v) + e;
        float s = 0.0f;
#pragma unroll 1
        for (int d = 0; d < A.C.D; ++d) s = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), s);
        const float p = __bfloat162float(__float2bfloat16_rn(ex2(s * A.scale_log2 - m)));
#pragma unroll 1
        for (int d = 0; d < dims; ++d) o[d] = fmaf(p, __bfloat162float(v[d0 + d]), o[d]);
    }
}

// Scores of a tile that the row does not see, all but the first `lim`, are set to -inf where they lie.  By a whole warp, from
// the first columns on that some row does not see.
__device__ __noinline__ void cut_scores(uint32_t s_addr, int lim) {
#pragma unroll 1
    for (int y = max(0, __reduce_min_sync(0xffffffffu, lim)) & ~15; y < kTile; y += 16) {
        uint32_t sc[16];
        ptx::tmem_ld16_bits(s_addr + y, sc);
        landed(sc);
#pragma unroll
        for (int z = 0; z < 16; ++z)
            if (y + z >= lim) sc[z] = 0xff800000u;
        ptx::tmem_st16_bits(s_addr + y, sc);
    }
    ptx::tmem_st_wait();
}

// 32 bytes, on a boundary of as many.
__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Maxima of a quarter of a tile's scores, in eight chains of three-input ones (one chain's latency would be the whole row's).
__device__ __forceinline__ void row_maxima(const uint32_t (&sc)[32], float (&tops)[8]) {
#pragma unroll
    for (int y = 0; y < 8; ++y) {
        const auto f = [&](int z) { return __uint_as_float(sc[y + 8 * z]); };
        tops[y] = max3(max3(tops[y], f(0), f(1)), f(2), f(3));
    }
}

__device__ __forceinline__ float row_maximum(const float (&tops)[8]) {
    return max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]), fmaxf(tops[6], tops[7]));
}

// 2^(c score + off) of a quarter of a tile's scores, rounded to bf16 in p; their sum, before the rounding, to `sum`.
__device__ __forceinline__ void probabilities(const uint32_t (&sc)[32], uint32_t *p, uint64_t c2, uint64_t off2, uint64_t (&sum)[2]) {
#pragma unroll
    for (int z = 0; z < 16; ++z) {
        float a, b;
        unpair(tat::fma2(pair(__uint_as_float(sc[2 * z]), __uint_as_float(sc[2 * z + 1])), c2, off2), a, b);
        a = ex2(a);
        b = ex2(b);
        sum[z & 1] = tat::add2(sum[z & 1], pair(a, b));
        p[z] = pack_bf16(a, b);
    }
}

template <int D>
__device__ __forceinline__ void soften(const PromptArgs &A, Misc *ms, uint32_t tmem, int tid_all) {
    using L = Lay<D>;
    const int s = L::NS == 2 ? tid_all >> 7 : 0, tid = tid_all & 127, warp = tid >> 5;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    const int tq = A.tokens / L::NS, RT = tq * A.GS;
    const int my_row = s * RT + tid;                           // row of the block's MT
    const float c = A.scale_log2;
    const Bars bars{ptx::smem_addr(ms)};
    // whole sectors at a time, where rows begin on them
    const bool wide = (reinterpret_cast<uintptr_t>(A.out) & 31) == 0 && A.C.D % 16 == 0;
    uint32_t seq = 0, outs = 0;                                // tiles taken, pieces put out
    int piece = 0;
    bool ok = true;
    const int own = s * tq + tid / A.GS;                       // the row's token of the block
    const int head = tid - (own - s * tq) * A.GS;              // and head of the group's part
    PieceReader reader;
    PieceInfo it, next;
    for (bool any = reader.next(ms, bars, &it, &ok); any; it = next, ++piece) {
        const PieceInfo &sp = it;
        const int n = s ? it.n[1] : it.n[0];
        const int g = it.part * A.GS + head;
        const bool on = tid < RT && it.q0 + own < it.cnt && g < A.G;
        const int64_t row = ((int64_t)it.first + it.q0 + own) * A.HQ + it.h * A.G + g;
        const bool whole = it.whole != 0;
        const int64_t part = (int64_t)it.chunk * 2 + (it.t0 == 0);
        const int see = on ? sp.all + own : INT32_MAX;         // keys that the row sees (no row: whatever there is)
        const int see_all = sp.all + s * tq;                   // that every row of the stream sees
        const bool warp_on = __any_sync(0xffffffffu, on);
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; ok && j < n; ++j, ++seq) {
            const int x = L::NS == 2 ? s : seq & 1, k0 = (it.t0 + j) * kTile;
            const uint32_t s_addr = lane_addr + L::col_s(x);
            ok = wait(bars.s_full(x), (L::NS == 2 ? seq : seq >> 1) & 1u, &ms->abort);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const auto hand_on = [&] {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if ((tid & 31) == 0) ptx::mbar_arrive(bars.p_full(x));
            };
            if (warp_on) {
                if (k0 + kTile > see_all) cut_scores(s_addr, see - k0);
                // One pass, 32 scores at a time, the next ones' load under way: the probabilities against the maximum so far and,
                // beside them, the tile's maximum.  They are kept until it is known that it has not grown too far.
                float tops[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) tops[y] = -INFINITY;
                const uint64_t c2 = pair(c, c);
                float s0 = 0.0f;
                bool move = j == 0;
                if (!move) {
                    uint32_t sa[32], sb[32], p[64];
                    uint64_t sum[2] = {0, 0};   // pairs of zeros
                    const float off = m == -INFINITY ? 0.0f : -m;
                    const uint64_t off2 = pair(off, off);
                    ptx::tmem_ld32_bits(s_addr, sa);
                    landed(sa);
                    ptx::tmem_ld32_bits(s_addr + 32, sb);
                    row_maxima(sa, tops);
                    probabilities(sa, p, c2, off2, sum);
                    landed(sb);
                    ptx::tmem_ld32_bits(s_addr + 64, sa);
                    row_maxima(sb, tops);
                    probabilities(sb, p + 16, c2, off2, sum);
                    landed(sa);
                    ptx::tmem_ld32_bits(s_addr + 96, sb);
                    row_maxima(sa, tops);
                    probabilities(sa, p + 32, c2, off2, sum);
                    landed(sb);
                    row_maxima(sb, tops);
                    probabilities(sb, p + 48, c2, off2, sum);
                    const float top = c * row_maximum(tops);
                    move = __any_sync(0xffffffffu, top > m + tat::kGrow);
                    if (!move) {
#pragma unroll
                        for (int y = 0; y < 64; y += 16) ptx::tmem_st16_bits(s_addr + y, p + y);
                        float s1;
                        unpair(tat::add2(sum[0], sum[1]), s0, s1);
                        s0 += s1;
                    }
                }
                if (move) {   // the maximum is to be moved: in two passes
                    uint32_t sc[32];
#pragma unroll 1
                    for (int y = 0; y < kTile; y += 32) {
                        ptx::tmem_ld32_bits(s_addr + y, sc);
                        landed(sc);
                        row_maxima(sc, tops);
                    }
                    const float top = c * row_maximum(tops), to = top > m + tat::kGrow ? top : m;
                    const float al = m == -INFINITY ? 0.0f : ex2(m - to);
                    l *= al;
                    m = to;
                    if (j > 0) {   // O holds the sums up to the tile before this one
                        // (with two streams they were issued before these scores, so they are done)
                        if (L::NS == 1) ok = wait(bars.pv_done(x ^ 1), ((seq - 1) >> 1) & 1u, &ms->abort);
                        if (!ok) break;
                        ptx::tc_fence_after_sync();
#pragma unroll 1
                        for (int y = 0; y < D; y += 32) {
                            ptx::tmem_ld32_bits(lane_addr + L::col_o(s) + y, sc);
                            landed(sc);
#pragma unroll
                            for (int z = 0; z < 32; ++z) sc[z] = __float_as_uint(__uint_as_float(sc[z]) * al);
                            ptx::tmem_st16_bits(lane_addr + L::col_o(s) + y, sc);
                            ptx::tmem_st16_bits(lane_addr + L::col_o(s) + y + 16, sc + 16);
                        }
                    }
                    const float off = m == -INFINITY ? 0.0f : -m;
                    const uint64_t off2 = pair(off, off);
                    uint64_t sum[2] = {0, 0};
#pragma unroll 1
                    for (int y = 0; y < kTile; y += 32) {
                        uint32_t p[16];
                        ptx::tmem_ld32_bits(s_addr + y, sc);
                        landed(sc);
                        probabilities(sc, p, c2, off2, sum);
                        ptx::tmem_st16_bits(s_addr + y / 2, p);   // over scores that have been read
                    }
                    float s1;
                    unpair(tat::add2(sum[0], sum[1]), s0, s1);
                    s0 += s1;
                }
                ptx::tmem_st_wait();
                hand_on();
                l += s0;
            } else {
                hand_on();
            }
        }
        if (!ok) break;
        any = reader.next(ms, bars, &next, &ok);   // (while the last sums run)
        if (!ok) break;
        if (n > 0) {
            ok = wait(bars.o_full(s), outs & 1u, &ms->abort);
            if (!ok) break;
            ++outs;
            ptx::tc_fence_after_sync();
            if (warp_on) {
                const bool removed = *(volatile int *)&ms->notes[piece % kNotes].piece == piece;
                const float inv = 1.0f / l;   // (no weight at all, every score -inf: infinite, and zeros times it are NaN)
#pragma unroll 1
                for (int d0 = 0; d0 < A.C.D; d0 += 32) {
                    uint32_t u[32];
                    ptx::tmem_ld32_bits(lane_addr + L::col_o(s) + d0, u);
                    landed(u);
                    const int dims = min(32, A.C.D - d0);
                    if (!on) continue;
                    if (removed) {   // rare: a copy of its own, so that u stays in registers
                        float g[32];
#pragma unroll
                        for (int y = 0; y < 32; ++y) g[y] = __uint_as_float(u[y]);
                        add_removed(A, ms, piece, it, sp.all, own, row, m, d0, dims, g);
#pragma unroll
                        for (int y = 0; y < 32; ++y) u[y] = __float_as_uint(g[y]);
                    }
                    const auto f = [&](int y) { return __uint_as_float(u[y]); };
                    if (whole) {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(A.out) + row * A.C.D + d0;
                        uint32_t w[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) w[y] = pack_bf16(f(2 * y) * inv, f(2 * y + 1) * inv);
                        if (wide && dims == 32) {
                            store32(out, w);
                            store32(out + 16, w + 8);
                        } else {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if (8 * y < dims)
                                    reinterpret_cast<uint4 *>(out)[y] = make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
                        }
                    } else {
                        float4 *po = A.part_o + (part * (A.C.D / 4) + d0 / 4) * A.MT + my_row;
#pragma unroll
                        for (int y = 0; y < 32; y += 4)
                            if (y < dims) po[(int64_t)(y / 4) * A.MT] = make_float4(f(y), f(y + 1), f(y + 2), f(y + 3));
                    }
                }
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if ((tid & 31) == 0) ptx::mbar_arrive(bars.o_empty(s));
        }
        if (on) {
            if (!whole) A.part_ml[part * A.MT + my_row] = make_float2(m, l);
            else if (A.lse) A.lse[row] = attn_lse(m, l);
        }
        __syncwarp();
        if ((tid & 31) == 0) *(volatile int *)&ms->done[tid_all >> 5] = piece + 1;
    }
}

template <int D>
__global__ void __launch_bounds__(Lay<D>::kThreads, 1)
prompt_attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ PromptArgs A) {
    using L = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *sm = smem_raw + pad;
    Misc *ms = reinterpret_cast<Misc *>(sm + L::kOffMisc);
    const uint32_t base = raw + pad;
    const int tid = threadIdx.x, warp = tid >> 5;
    uint32_t have;
    asm("mov.u32 %0, %dynamic_smem_size;" : "=r"(have));
    if (pad + L::kOffMisc + sizeof(Misc) > have) {   // the segment does not start where it always has
        grid_dep_wait();
        if (tid == 0) {
            atomicOr(A.C.status, GDN_SPEC_ST_TIMEOUT);
            for (int w = 0; w < A.waves; ++w) prompt_note(A, PromptWalk(), 1, w);   // the join finds empty chunks
        }
        return;
    }
    if (tid == 0) {
        const auto init = [](uint64_t &b, uint32_t n) { ptx::mbar_init(ptx::smem_addr(&b), n); };
        for (int i = 0; i < L::NST; ++i) {
            init(ms->full[i], 1);
            init(ms->empty[i], L::NS);   // warps that use the stage
            init(ms->clean[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            init(ms->piece_full[i], 1);
            init(ms->piece_empty[i], L::NS * 4 + 2 + L::kProducers);   // warps that read it
        }
        for (int i = 0; i < 2; ++i) {
            init(ms->q_full[i], 1);
            init(ms->q_empty[i], 1);
            init(ms->s_full[i], 1);
            init(ms->p_full[i], 4);
            init(ms->o_full[i], 1);
            init(ms->o_empty[i], 4);
            init(ms->pv_done[i], 1);
            init(ms->turn[i], 1);
            init(ms->drain[i], 1);
        }
        for (int i = 0; i < kNotes; ++i) ms->notes[i].piece = -1;
        for (int i = 0; i < 8; ++i) ms->done[i] = 0;
        ms->abort = 0;
        ptx::mbar_init_fence();
        ptx::prefetch_tmap(&mq);
        ptx::prefetch_tmap(&mk);
        ptx::prefetch_tmap(&mv);
    }
    if (warp == 0) ptx::tmem_alloc(ptx::smem_addr(&ms->tmem), kTmemCols);
    grid_dep_wait();   // nothing in global memory was touched so far
    const PromptPlan plan = prompt_plan<L::kThreads>(A, &ms->scratch);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = ms->tmem;

    if (warp < L::NS * 4) {
        // while the first tile is on its way
        prompt_dead_tokens<__nv_bfloat16>(A, plan.ascends(), tid, L::NS * 128);
        soften<D>(A, ms, tmem, tid);
    } else {
        const int role = warp - L::NS * 4;
        if (role == 0) {
            produce<D, true, L::kProducers == 1>(A, &mq, &mk, &mv, ms, base, plan);
        } else if (L::kProducers == 2 && role == 4) {
            produce<D, false, true>(A, &mq, &mk, &mv, ms, base, plan);
        } else if (role == 3) {
            clean<D>(A, ms, sm);
        } else if (L::NS == 2) {
            multiply_stream<D>(A, ms, base, tmem, role - 1);
        } else if (role == 1) {
            multiply_scores<D>(A, ms, base, tmem);
        } else {
            multiply_sums<D>(A, ms, base, tmem);
        }
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

template <int D>
cudaError_t run(const PromptArgs &A, cudaStream_t st) {
    using L = Lay<D>;
    static_assert(L::kOffMisc + sizeof(Misc) <= kSmemMax && L::NST <= kMaxStages, "shared memory");
    // room to reach a 1024-byte boundary (the dynamic segment starts on one: there is no static one)
    constexpr size_t need = L::kOffMisc + sizeof(Misc) + 1024;
    constexpr size_t smem = need < (size_t)kSmemMax ? need : (size_t)kSmemMax;
    static KernelSetup setup;
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)prompt_attn_tc_kernel<D>, smem, &sms);
    if (e != cudaSuccess) return e;
    const cuuint64_t rows = (cuuint64_t)A.C.n_layers * A.C.num_pages * A.C.HKV * A.C.P, dims = A.C.D;
    // Keys and values as (64 dims, token rows, blocks of 64 dims) where a box can hold all of a stage's blocks (they land
    // one after another), else as (dims, token rows, 1) with a box for each block; dims past the head's are filled with
    // zeros.
    const auto map_kv = [&](CUtensorMap *map, const void *p, bool whole, int tokens, uint32_t blocks) {
        const cuuint64_t size[3] = {whole ? 64 : dims, rows, whole ? dims / 64 : 1}, stride[2] = {dims, 64};
        const cuuint32_t box[3] = {64, (cuuint32_t)(A.C.P < tokens ? A.C.P : tokens), whole ? blocks : 1u};
        return tat::bf16_map(map, p, 3, size, stride, box);
    };
    const int tq = A.tokens / L::NS;
    const cuuint64_t q_dims[3] = {dims, (cuuint64_t)A.HQ, (cuuint64_t)A.N}, q_stride[2] = {dims, (cuuint64_t)A.HQ * dims};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)A.GS, (cuuint32_t)(tq < A.N ? tq : A.N)};
    CUtensorMap mq, mk, mv;
    if (!map_kv(&mk, A.C.k, A.k_whole, kTile, L::kKBlocks) || !map_kv(&mv, A.C.v, A.v_whole, L::kVRows, L::kVBlocks) ||
        !tat::bf16_map(&mq, A.q, 3, q_dims, q_stride, q_box))
        return cudaErrorInvalidValue;
    return launch_dependent(prompt_attn_tc_kernel<D>, dim3(A.groups), dim3(L::kThreads), smem, st, mq, mk, mv, A);
}

}  // namespace pat

// Rows of the pool are coordinates of a copy.
bool prompt_attn_tc_supported(const KvArgs &C) { return (int64_t)C.n_layers * C.num_pages * C.HKV * C.P <= INT32_MAX; }

// The cut of the work: a stream's query tile holds whole tokens, as many as fit in 128 rows.
void prompt_attn_tc_cut(PromptArgs *A, int sms) {
    const int streams = A->C.D > 128 ? 1 : 2;
    A->HS = (A->G + pat::kRows - 1) / pat::kRows;
    A->GS = (A->G + A->HS - 1) / A->HS;
    A->tokens = streams * (pat::kRows / A->GS);
    A->MT = A->tokens * A->GS;
    A->log_tn = pat::kLogTile;
    A->k_whole = A->C.P >= pat::kTile && A->C.D % 64 == 0 && A->C.D != 192;
    A->v_whole = A->C.P >= pat::kTile / (A->C.D > 128 ? 2 : 1) && A->C.D % 64 == 0 && A->C.D != 192;
    A->groups = sms;
    // several waves where a layer of the pool is more than one wave's, and rows have blocks enough to read it again
    const int64_t pool = (int64_t)A->C.num_pages * A->C.P * A->C.HKV * A->C.D * 4;
    const int64_t waves = pool / kPromptWaveBytes + 1;
    A->waves = A->N < 2 * (int64_t)A->tokens * A->B ? 1 : waves < kPromptWaves ? (int)waves : kPromptWaves;
    A->gap = (streams == 2 ? 3 : 4) * pat::kTile;
}

cudaError_t launch_prompt_attn_tc(const PromptArgs &A, cudaStream_t st) {
    const cudaError_t e = A.C.D <= 64 ? pat::run<64>(A, st) : A.C.D <= 128 ? pat::run<128>(A, st) : pat::run<256>(A, st);
    return e != cudaSuccess ? e : launch_prompt_join(A, true, st);
}

}  // namespace gdnspec
