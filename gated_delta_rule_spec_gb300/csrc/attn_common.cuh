// attn_common.cuh -- how the tree attention's work is cut and put together
// again; shared by its kernels and by the kernel that joins split rows.
//
// An item is one (batch row, kv head): its query rows are the row's cnt drafted
// tokens times the G heads of the group (row r is token r / G, head r % G), cut into
// query tiles of MT rows, and it is a run of `tiles` key/value tiles of TN tokens.
// Items stand in one line, rows first, each behind a gap of as many tiles as an item
// costs besides its tiles, and the line is cut into equal chunks, one for each group
// of NQT blocks (one block per query tile of the item, so the blocks that read the
// same keys and values run side by side and share them in L2).  So ragged rows, few
// rows with long contexts and many short ones all spread evenly over the machine,
// and every block finds its chunk from the lengths on the device: nothing about
// them is known on the host.  A chunk that
// starts or ends inside an item leaves an unnormalised piece in the workspace (at
// most two a block), and the join kernel merges an item's pieces in order, so the
// result does not depend on timing.
#pragma once

#include "kv_common.cuh"

namespace gdnspec {

struct AttnArgs {
    KvArgs C;
    int layer, B, T, HQ, G;
    const int32_t *slot_idx;
    const uint64_t *tree_mask;
    const int32_t *tree_len;
    float scale_log2;          // scale * log2(e): probabilities are powers of two
    const void *q;
    void *out;
    float *lse;
    float4 *part_o;            // [groups * NQT][2][D / 4][MT] unnormalised sums of a piece
    float2 *part_ml;           // [groups * NQT][2][MT] (maximum in log2 units, sum)
    struct AttnCut *cuts;      // [groups] where each chunk starts, for the join
    int TN, MT, NQT, groups, min_chunk, gap;
    bool whole;                // tensor-core kernel: a copy holds all dims of a tile
    uint32_t wait_limit;
};

struct AttnRow {
    int slot, len, cnt;        // cnt = 0: nothing to compute
};

__device__ __forceinline__ AttnRow attn_row(const AttnArgs &A, int b, uint32_t *bits) {
    AttnRow r;
    r.slot = A.slot_idx[b];
    r.cnt = A.tree_len ? A.tree_len[b] : A.T;
    r.len = kv_row(A.C, r.slot, r.cnt, A.T, bits);
    if (r.len < 0) r.len = r.cnt = 0;
    return r;
}

__device__ __forceinline__ int attn_tiles(const AttnArgs &A, const AttnRow &r) {
    return r.cnt > 0 ? (int)(((int64_t)r.len + r.cnt + A.TN - 1) / A.TN) : 0;
}

// Length of a row's part of the line.
__device__ __forceinline__ int attn_span(const AttnArgs &A, const AttnRow &r) {
    const int tiles = attn_tiles(A, r);
    return tiles > 0 ? (tiles + A.gap) * A.C.HKV : 0;
}

// A place of the line: the row it is in, and where in the row's part.
struct AttnPlan {
    int total, chunk;          // length of the line and of a chunk
    int b, off;                // of the asked place (b = -1: past the end)
};

constexpr int kAttnScratch = 34;   // ints of shared memory for attn_plan

// Sum over the block of x; *before: of the threads below.
template <int THREADS>
__device__ __forceinline__ int attn_scan(int x, int *scratch, int *before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int sum = 0, base = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int s = scratch[w];
        if (w < warp) base += s;
        sum += s;
    }
    *before = base + inc - x;
    __syncthreads();
    return sum;
}

// By all threads of a block: the line's length and the place
// group * chunk.  `report`: record the rows' status bits.
template <int THREADS>
__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs &A, int group, bool report, int *scratch) {
    int *const place = scratch + 32;
    AttnPlan p;
    const int tid = threadIdx.x;
    p.total = 0;
    int mine = 0, before = 0;   // of the first THREADS rows
    for (int b0 = 0; b0 < A.B; b0 += THREADS) {
        int x = 0, ex;
        if (b0 + tid < A.B) {
            uint32_t bits;
            const AttnRow r = attn_row(A, b0 + tid, &bits);
            if (bits && report) atomicOr(A.C.status, bits);
            x = attn_span(A, r);
        }
        const int sum = attn_scan<THREADS>(x, scratch, &ex);
        if (b0 == 0) { mine = x; before = ex; }
        p.total += sum;
    }
    p.chunk = max(A.min_chunk, (p.total + A.groups - 1) / A.groups);
    const int64_t at = (int64_t)group * p.chunk;
    if (tid == 0) place[0] = -1;
    __syncthreads();
    if (at < p.total) {
        int base = 0;
        for (int b0 = 0; b0 < A.B; b0 += THREADS) {
            int x = mine, ex = before;
            if (b0 > 0) {
                x = 0;
                if (b0 + tid < A.B) {
                    uint32_t bits;
                    x = attn_span(A, attn_row(A, b0 + tid, &bits));
                }
            }
            int sum = 0;
            if (A.B > THREADS) {
                int e2;
                sum = attn_scan<THREADS>(x, scratch, &e2);
                ex = e2;
            }
            if (x > 0 && base + ex <= at && at < base + ex + x) {
                place[0] = b0 + tid;
                place[1] = (int)(at - base - ex);
            }
            base += sum;
        }
    }
    __syncthreads();
    p.b = place[0];
    p.off = place[1];
    return p;
}

// The pieces of a chunk, one after another.  Every thread that walks does so alone.
struct AttnPiece {
    int b, slot, len, cnt, h;
    int t0, t1, tiles;         // key/value tiles [t0, t1) of the item's `tiles`
    int side;                  // which of the block's two pieces it would be kept as: 1 if it starts its item
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Keeps the row between its heads: a row's counts are three dependent loads.
struct AttnWalk {
    AttnRow row;
    int b, h, t, tiles, left;   // next tile; left: what is left of the chunk
    __device__ __forceinline__ void load(const AttnArgs &A) {
        uint32_t bits;
        row = attn_row(A, b, &bits);
        tiles = attn_tiles(A, row);
    }
    __device__ __forceinline__ bool next(const AttnArgs &A, AttnPiece *piece) {
        if (left <= 0) return false;
        if (t == tiles) {
            t = 0;
            ++h;
            left -= A.gap;
            if (left <= 0) return false;
        }
        if (h >= A.C.HKV) {
            h = 0;
            do {
                if (++b >= A.B) return false;
                load(A);
            } while (tiles == 0);
        }
        piece->b = b;
        piece->slot = row.slot;
        piece->len = row.len;
        piece->cnt = row.cnt;
        piece->h = h;
        piece->t0 = t;
        piece->t1 = min(tiles, t + left);
        piece->tiles = tiles;
        piece->side = t == 0;
        left -= piece->t1 - t;
        t = piece->t1;
        return true;
    }
};

// Where a chunk starts, noted by the group's first block.
struct __align__(16) AttnCut {
    int b, h, t, tiles;        // row (-1: the chunk is empty), kv head, tile of the item's `tiles`
    int cnt, chunk, pad[2];    // the row's tokens, tiles of a chunk
};

__device__ __forceinline__ void attn_note(const AttnArgs &A, int group, bool any, const AttnPiece &pc, int chunk) {
    A.cuts[group] = any ? AttnCut{pc.b, pc.h, pc.t0, pc.tiles, pc.cnt, chunk, {0, 0}} : AttnCut{-1, 0, 0, 0, 0, chunk, {0, 0}};
}

__device__ __forceinline__ AttnWalk attn_walk(const AttnArgs &A, const AttnPlan &p, int group) {
    AttnWalk w;
    w.left = 0;
    if (p.b < 0) return w;
    w.b = p.b;
    w.load(A);
    w.h = p.off / (w.tiles + A.gap);
    const int in_item = p.off - w.h * (w.tiles + A.gap) - A.gap;   // < 0: in the gap before the item
    w.t = max(in_item, 0);
    w.left = min(in_item, 0) + (int)min((int64_t)p.chunk, (int64_t)p.total - (int64_t)group * p.chunk);
    return w;
}

// Nodes that token t attends to, as bits.
__device__ __forceinline__ uint64_t attn_mask(const AttnArgs &A, int b, int t) {
    return A.tree_mask ? A.tree_mask[(int64_t)b * A.T + t] : (2ull << t) - 1;
}

__device__ __forceinline__ int64_t attn_out_row(const AttnArgs &A, int b, int h, int r) {
    const int t = r / A.G, g = r - t * A.G;
    return ((int64_t)b * A.T + t) * A.HQ + h * A.G + g;
}

// Rows that nothing computes (tokens past cnt, rows that were refused): zeros, and
// an lse of -inf.  By `threads` threads of each block, the batch rows in turn.
template <typename IO>
__device__ __forceinline__ void attn_dead_rows(const AttnArgs &A, int block, int blocks, int thread, int threads) {
    for (int b = block; b < A.B; b += blocks) {
        uint32_t bits;
        const AttnRow r = attn_row(A, b, &bits);
        const int64_t row0 = ((int64_t)b * A.T + r.cnt) * A.HQ, rows = (int64_t)(A.T - r.cnt) * A.HQ;
        float4 *o = reinterpret_cast<float4 *>(static_cast<IO *>(A.out) + row0 * A.C.D);
        const int64_t n = rows * A.C.D * sizeof(IO) / 16;
        for (int64_t i = thread; i < n; i += threads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (A.lse)
            for (int64_t i = thread; i < rows; i += threads) A.lse[row0 + i] = -INFINITY;
    }
}

__device__ __forceinline__ float attn_lse(float m2, float l) {
    return l > 0.0f ? (m2 + log2f(l)) * 0.6931471805599453f : (l == 0.0f ? -INFINITY : NAN);
}

// Joins the pieces of split items: block (g, query tile, part) takes the item
// whose first inner cut is the end of chunk g - 1.
cudaError_t launch_attn_join(const AttnArgs &A, bool bf16, cudaStream_t stream);

}  // namespace gdnspec
