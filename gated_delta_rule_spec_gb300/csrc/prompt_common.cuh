// prompt_common.cuh -- how the work of the attention of packed prompts is cut and put
// together again; shared by its kernels and by the kernel that joins split items.
//
// Row b of a call owns tokens starts[b] .. starts[b + 1] of the packed tensors.  Its item
// (h, i) is one kv head h and one block i of `tokens` consecutive tokens: the block's
// tokens times the GS query heads of the group are the rows of the products (row r is
// token r / GS, head r % GS), and its keys are the committed ones and those of the
// tokens up to the block's last.  A group of more heads than a block has rows goes in HS
// parts, each like a kv head of its own.
//
// Items stand in one line, rows first, then heads, then blocks; an item's length is its keys
// plus `gap`, what it costs besides them, so a row's part of the line is an arithmetic
// series and both directions (the place where item i starts, the item at a place) are
// closed forms.  The line is cut into equal chunks, `waves` of them for each block of the grid,
// which finds its own from the counts on the device.  So one long prompt, many short ones and
// single tokens behind long contexts all spread evenly over the machine, and nothing
// about the lengths is known on the host.  Chunk w * groups + g is block g's in wave w: where all
// rows' keys and values are more than L2 holds, the blocks go through them together, a part that
// L2 holds at a time (4 rows of 499 to 1024 tokens behind 19751 to 30000, 64 heads on 8 of 128, 400 MB: 10.0 GB read
// from HBM and 1824 us in one wave, 2.4 GB and 1680 us in four).  A cut inside an item falls on a key tile and
// leaves unnormalised pieces in the workspace (at most two a chunk), which the join
// kernel merges in order: the result does not depend on timing.
#pragma once

#include "attn_common.cuh"

namespace gdnspec {

struct PromptArgs {
    KvArgs C;
    int layer, B, N, HQ, G;
    int GS, HS;                // heads of a part of a group, parts of a group
    const int32_t *slot_idx, *starts;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    const void *q;
    void *out;
    float *lse;
    float4 *part_o;            // [chunks][2][D / 4][MT] unnormalised sums of a piece
    float2 *part_ml;           // [chunks][2][MT] (maximum in log2 units, sum)
    struct PromptCut *cuts;    // [chunks] where each chunk starts, for the join
    int log_tn, MT, tokens;    // keys of a tile (2^log_tn); rows and tokens of a block
    int groups, waves, gap;    // blocks; chunks of a block at most
    bool k_whole, v_whole;     // tensor-core kernel: one copy holds all dims of a stage
    uint32_t wait_limit;
};

struct PromptRow {
    int slot, len, cnt;        // cnt = 0: nothing to compute
    int first, owned;          // its tokens in the packed tensors
};

__device__ __forceinline__ bool prompt_range(const PromptArgs &A, int first, int end) { return first >= 0 && end >= first && end <= A.N; }

// Whether a row before row b that is a range reaches past b's first token.  Only where some row is no range: if all are,
// starts ascends.  Out of line: inside the append it costs what its loads are ordered by (36101 tokens of 32 + 2 x 8 heads
// of 128: 200 us, 175 so).
__device__ __noinline__ inline bool prompt_overlaps(const PromptArgs &A, int b, int first) {
    for (int e = 0; e < b; ++e) {
        const int end = A.starts[e + 1];
        if (end > first && prompt_range(A, A.starts[e], end)) return true;
    }
    return false;
}

// ascends: every row is a range.
__device__ __forceinline__ PromptRow prompt_row(const PromptArgs &A, int b, bool ascends, uint32_t *bits) {
    PromptRow r;
    r.slot = A.slot_idx[b];
    r.first = A.starts[b];
    const int end = A.starts[b + 1];
    *bits = 0;
    // no range of tokens, or tokens that are another's: there is nothing that could be written
    if (!prompt_range(A, r.first, end) || (!ascends && prompt_overlaps(A, b, r.first))) {
        *bits = GDN_SPEC_ST_ACCEPT_RANGE;
        r.first = r.owned = r.len = r.cnt = 0;
        return r;
    }
    r.cnt = r.owned = end - r.first;
    r.len = kv_row(A.C, r.slot, r.cnt, r.cnt, bits);
    if (r.len < 0) r.len = r.cnt = 0;
    return r;
}

// The line of one row: `blocks` items for each of its heads, block i starting `before(i)` behind the head's start.
struct PromptLine {
    int blocks;
    int64_t step, head;        // an item's length without its own tokens; a head's
    int tokens;
    __device__ __forceinline__ PromptLine(const PromptArgs &A, const PromptRow &r) : tokens(A.tokens) {
        blocks = (r.cnt + A.tokens - 1) / A.tokens;
        step = (int64_t)r.len + A.gap;
        head = blocks ? before(blocks - 1) + step + r.cnt : 0;
    }
    __device__ __forceinline__ int64_t before(int64_t i) const { return i * step + tokens * (i * (i + 1) / 2); }
    // the item at place `off` of the head
    __device__ __forceinline__ int at(int64_t off) const {
        // tokens / 2 i^2 + b i = off, in the form without a difference; the loops take what fp32 is off by
        const float b = (float)step + 0.5f * tokens;
        int i = (int)fminf(2.0f * (float)off / (b + sqrtf(b * b + 2.0f * tokens * (float)off)), 2.0e9f);
        i = max(0, min(i, blocks - 1));
        while (i > 0 && before(i) > off) --i;
        while (i + 1 < blocks && before(i + 1) <= off) ++i;
        return i;
    }
};

__device__ __forceinline__ int64_t prompt_span(const PromptArgs &A, const PromptRow &r) {
    return PromptLine(A, r).head * A.C.HKV * A.HS;
}

// One item: what it covers and where it stands in the line.
struct PromptItem {
    int b, slot, len, cnt, first;
    int h, part, q0;           // kv head, part of its group, the block's first token of the row
    int keys, tiles;
    int64_t pos;               // its place in the line
    // The tile on which a cut at this place of the line falls.
    __device__ __forceinline__ int tile_at(const PromptArgs &A, int64_t place) const {
        const int64_t off = place - pos - A.gap;
        return off <= 0 ? 0 : off >= keys ? tiles : (int)(off >> A.log_tn);
    }
};

// Where a chunk starts, noted by its block for the join; item.b = -1: past the end.
struct __align__(16) PromptCut {
    PromptItem item;
    int64_t chunk;
};

constexpr int kPromptWaves = 4;                 // at most
constexpr int64_t kPromptWaveBytes = 96 << 20;  // keys and values of a wave, of rows with several blocks
constexpr int kPromptWaveKeys = 2048;           // of a chunk at least, where there are several of a block

struct PromptScratch {
    int64_t sums[32];
    int64_t off[kPromptWaves];   // where the block's chunks start: the place in the row's part
    int b[kPromptWaves];         // and the row (-1: past the end)
    int ascends;                 // whether the entries of starts do
};

struct PromptPlan {
    int64_t total, chunk;      // length of the line and of a chunk
    const PromptScratch *at;   // the chunks' starts
    __device__ __forceinline__ bool ascends() const { return at->ascends != 0; }
};

// Sum over the block of x; *before: of the threads below.
template <int THREADS>
__device__ __forceinline__ int64_t prompt_scan(int64_t x, PromptScratch *sc, int64_t *before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sc->sums[warp] = inc;
    __syncthreads();
    int64_t sum = 0, base = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int64_t s = sc->sums[w];
        if (w < warp) base += s;
        sum += s;
    }
    *before = base + inc - x;
    __syncthreads();
    return sum;
}

// By all threads of a block: the line's length, and the rows at which its chunks start; false: ASCENDS is not so.
// The grid's first block records the rows' status bits.
template <int THREADS, bool ASCENDS>
__device__ __forceinline__ bool prompt_lay_out(const PromptArgs &A, PromptScratch *sc, PromptPlan *plan) {
    PromptPlan &p = *plan;
    const int tid = threadIdx.x;
    p.total = 0;
    p.at = sc;
    int64_t mine = 0, before = 0, keys = 0;   // of the first THREADS rows; of this thread's rows
    uint32_t all = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < A.B; b0 += THREADS) {
        int64_t x = 0, ex;
        if (b0 + tid < A.B) {
            uint32_t bits;
            const PromptRow r = prompt_row(A, b0 + tid, ASCENDS, &bits);
            all |= bits;
            x = prompt_span(A, r);
            if (r.cnt > 2 * A.tokens) keys += r.len + r.cnt;
        }
        const int64_t sum = prompt_scan<THREADS>(x, sc, &ex);
        if (b0 == 0) { mine = x; before = ex; }
        p.total += sum;
    }
    if (ASCENDS && __syncthreads_or(all & GDN_SPEC_ST_ACCEPT_RANGE)) return false;
    if (all && blockIdx.x == 0) atomicOr(A.C.status, all);
    if (tid == 0) sc->ascends = ASCENDS;
    int64_t waves = 1;
    if (A.waves > 1) {
        int64_t ex;
        keys = prompt_scan<THREADS>(keys, sc, &ex);
        waves = min((int64_t)A.waves, keys * A.C.HKV * A.C.D * 4 / kPromptWaveBytes + 1);   // (16-bit keys and values)
    }
    // a chunk is a tile at least, so that cuts inside an item fall on different tiles
    p.chunk = (p.total + A.groups - 1) / A.groups;
    if (waves > 1) p.chunk = max((p.total + A.groups * waves - 1) / (A.groups * waves), min(p.chunk, (int64_t)kPromptWaveKeys));
    p.chunk = max((int64_t)1 << A.log_tn, p.chunk);
    if (tid < kPromptWaves) sc->b[tid] = -1;
    __syncthreads();
    int64_t base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < A.B; b0 += THREADS) {
        int64_t x = mine, ex = before;
        if (b0 > 0) {
            x = 0;
            if (b0 + tid < A.B) {
                uint32_t bits;
                x = prompt_span(A, prompt_row(A, b0 + tid, ASCENDS, &bits));
            }
        }
        int64_t sum = 0;
        if (A.B > THREADS) {
            int64_t e2;
            sum = prompt_scan<THREADS>(x, sc, &e2);
            ex = e2;
        }
#pragma unroll 1
        for (int w = 0; w < A.waves; ++w) {
            const int64_t at = ((int64_t)w * A.groups + blockIdx.x) * p.chunk;
            if (x > 0 && base + ex <= at && at < base + ex + x) {
                sc->b[w] = b0 + tid;
                sc->off[w] = at - base - ex;
            }
        }
        base += sum;
    }
    __syncthreads();
    return true;
}

template <int THREADS>
__device__ __noinline__ PromptPlan prompt_plan_no_order(const PromptArgs &A, PromptScratch *sc) {
    PromptPlan p;
    prompt_lay_out<THREADS, false>(A, sc, &p);
    return p;
}

template <int THREADS>
__device__ __forceinline__ PromptPlan prompt_plan(const PromptArgs &A, PromptScratch *sc) {
    PromptPlan p;
    return prompt_lay_out<THREADS, true>(A, sc, &p) ? p : prompt_plan_no_order<THREADS>(A, sc);
}

// The pieces of a block's chunk, one after another, for whoever walks.
struct PromptPiece {
    PromptItem it;
    int t0, t1;                // key tiles [t0, t1) of the item's
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.tiles; }
    // which of the block's two pieces it would be kept as: 1 if it starts its item
    __device__ __forceinline__ int side() const { return t0 == 0; }
    // keys that the tokens before `token` of the row attend to at most
    __device__ __forceinline__ int keys_to(int token) const { return it.len + min(it.cnt, token); }
};

struct PromptWalk {
    PromptItem it;
    int hp, i, blocks;         // head times parts of it, block, the row's blocks
    int64_t start, end;        // the chunk
    bool live;

    __device__ __forceinline__ void load(const PromptArgs &A, const PromptPlan &p) {
        uint32_t bits;
        const PromptRow r = prompt_row(A, it.b, p.ascends(), &bits);
        it.slot = r.slot, it.len = r.len, it.cnt = r.cnt, it.first = r.first;
        blocks = (r.cnt + A.tokens - 1) / A.tokens;
    }
    __device__ __forceinline__ void set(const PromptArgs &A) {
        it.h = A.HS == 1 ? hp : hp / A.HS;
        it.part = A.HS == 1 ? 0 : hp - it.h * A.HS;
        it.q0 = i * A.tokens;
        it.keys = it.len + min(it.cnt, it.q0 + A.tokens);
        it.tiles = (it.keys + (1 << A.log_tn) - 1) >> A.log_tn;
    }
    __device__ __forceinline__ PromptWalk() : live(false) {}
    // Through the block's chunk of wave w.
    __device__ __forceinline__ PromptWalk(const PromptArgs &A, const PromptPlan &p, int w) {
        live = p.at->b[w] >= 0;
        if (!live) return;
        start = ((int64_t)w * A.groups + blockIdx.x) * p.chunk;
        end = min(p.total, start + p.chunk);
        it.b = p.at->b[w];
        uint32_t bits;
        const PromptRow r = prompt_row(A, it.b, true, &bits);   // (a row that has items)
        it.slot = r.slot, it.len = r.len, it.cnt = r.cnt, it.first = r.first;
        const PromptLine line(A, r);
        const int64_t off = p.at->off[w];
        blocks = line.blocks;
        hp = (int)(off / line.head);
        const int64_t in = off - hp * line.head;
        i = line.at(in);
        it.pos = start - (in - line.before(i));
        set(A);
    }
    __device__ __forceinline__ bool next(const PromptArgs &A, const PromptPlan &p, PromptPiece *pc) {
        while (live) {
            pc->it = it;
            pc->t0 = it.tile_at(A, start);
            pc->t1 = it.tile_at(A, end);
            it.pos += it.keys + A.gap;
            if (it.pos >= end) {
                live = false;
            } else {
                if (++i == blocks) {
                    i = 0;
                    if (++hp == A.C.HKV * A.HS) {
                        hp = 0;
                        do {
                            if (++it.b >= A.B) {   // not reached while the line is as planned
                                live = false;
                                break;
                            }
                            load(A, p);
                        } while (it.cnt == 0);
                    }
                }
                if (live) set(A);
            }
            if (pc->t0 < pc->t1) return true;
        }
        return false;
    }
};

// The note of the block's chunk of wave w; by one thread, before the walk begins.
__device__ __forceinline__ void prompt_note(const PromptArgs &A, const PromptWalk &walk, int64_t chunk, int w) {
    PromptCut c;
    if (walk.live) c.item = walk.it;
    else c.item.b = -1;
    c.chunk = chunk;
    A.cuts[w * A.groups + blockIdx.x] = c;
}

// Row of the output for row r of an item's block, and whether the row is one.
__device__ __forceinline__ int64_t prompt_out_row(const PromptArgs &A, const PromptItem &it, int r, bool *on) {
    const int t = r / A.GS, g = it.part * A.GS + r - t * A.GS;
    *on = t < A.tokens && it.q0 + t < it.cnt && g < A.G;
    return ((int64_t)it.first + it.q0 + t) * A.HQ + it.h * A.G + g;
}

// The row that owns `token`, if one does; by a whole warp.  In [0, B) always.  Where starts ascends: the last one that
// starts at or before it, 32 rows looked at in one step.  Else the first row that is a range with it inside (a later one
// overlaps that row).
__device__ __forceinline__ int prompt_owner(const PromptArgs &A, int token, bool ascends) {
    const int lane = threadIdx.x & 31, B = A.B;
    const int32_t *const starts = A.starts;
    if (!ascends) {
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int b = b0 + lane;
            const bool in = b < B && starts[b] <= token && token < starts[b + 1] && prompt_range(A, starts[b], starts[b + 1]);
            const unsigned some = __ballot_sync(0xffffffffu, in);
            if (some) return b0 + __ffs(some) - 1;
        }
        return 0;
    }
    int lo = 0, n = B;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && starts[at] <= token);
        const int k = max(0, 31 - __clz(below));   // the last lane that starts at or before it (rows ascend)
        const int end = lo + n;
        lo += k * step;
        n = min(step, end - lo);
    }
    return lo;
}

// Tokens of rows that nothing computes (padding rows, rows that were refused): zeros, and an lse of -inf.  By `threads`
// threads (whole warps) of each block; every block takes an equal share of the packed tokens.
template <typename IO>
__device__ __noinline__ void prompt_dead_tokens(const PromptArgs &A, bool ascends, int thread, int threads) {
    const int n0 = (int)((int64_t)A.N * blockIdx.x / gridDim.x), n1 = (int)((int64_t)A.N * (blockIdx.x + 1) / gridDim.x);
    if (n0 >= n1) return;
    for (int b = ascends ? prompt_owner(A, n0, true) : 0; b < A.B; ++b) {
        if (A.starts[b] >= n1 || A.starts[b + 1] <= n0) {   // none of its tokens are this block's
            if (ascends && A.starts[b] >= n1) break;
            continue;
        }
        uint32_t bits;
        const PromptRow r = prompt_row(A, b, ascends, &bits);
        if (r.cnt || !r.owned) continue;
        const int64_t t0 = max(n0, r.first), t1 = min(n1, r.first + r.owned);
        float4 *o = reinterpret_cast<float4 *>(static_cast<IO *>(A.out) + t0 * A.HQ * A.C.D);
        const int64_t n = (t1 - t0) * A.HQ * A.C.D * (int64_t)sizeof(IO) / 16;
        for (int64_t i = thread; i < n; i += threads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (A.lse)
            for (int64_t i = thread; i < (t1 - t0) * A.HQ; i += threads) A.lse[t0 * A.HQ + i] = -INFINITY;
    }
}

cudaError_t launch_prompt_join(const PromptArgs &A, bool bf16, cudaStream_t stream);

}  // namespace gdnspec
