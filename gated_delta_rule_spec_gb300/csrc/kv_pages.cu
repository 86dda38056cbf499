// kv_pages.cu -- the pages of the softmax-attention cache: reserve, fork,
// commit, free.
//
// Free pages are a bitmap, one bit per page, and the pages handed out are the
// free ones of lowest number, in row order.  So the tables depend only on the
// sequence of calls: releasing a page is an atomic decrement of its holders and,
// by the holder that reaches zero, an atomic OR of its bit, and neither's order
// shows in the result.  A free list (a stack or a queue) would need the released
// pages sorted to be as repeatable.
//
// The allocation is one block: it reads the whole bitmap once (128 KB for a
// million pages) to count what is free, then walks it in slices of 1024 words
// until the rows' demand is met.  Within a slice every page that is handed out has a
// thread of its own, which finds its bit and its row by bisection (a thread per
// word took 16 us for 512 pages, this takes 6 us).
// Everything that moves key/value rows is a launch of its own over the whole
// machine, bound by HBM.
#include "kv_common.cuh"
#include "launch_setup.cuh"

namespace gdnspec {

constexpr int kAllocThreads = 1024;
constexpr int kAllocRows = 8192;      // rows of one reserve or fork: their running demand is kept in shared memory
constexpr int kCopyThreads = 256;
constexpr int kMoveMaxT = 1024;       // window of a commit with a path
// Table entries (rows times columns) of a fork that the allocating block looks at itself; beyond them a launch of its
// own does.  What looking at them adds to a fork, in the block and as a launch: 32 rows of 126 columns 0.9 and 2.3 us,
// 128 of 65 1.8 and 1.4, 256 of 126 4.2 and 1.9, 64 of 8189 25 and 3.
constexpr int64_t kForkInline = 6 << 10;

// Exclusive prefix sum over the block's threads; *total is the block's sum.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = lane < nw ? warp_sums[lane] : 0;
        int winc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, winc, o);
            if (lane >= o) winc += y;
        }
        warp_sums[lane] = winc - w;
        if (lane == 31) warp_sums[32] = winc;
    }
    __syncthreads();
    const int r = warp_sums[warp] + inc - x;
    *total = warp_sums[32];
    __syncthreads();   // warp_sums may be written again
    return r;
}

// What a row asks for: pages to add to `slot` behind its first `have` ones.
struct Demand {
    int slot, have, need;
    bool ok;
};

template <bool FORK>
__device__ __forceinline__ Demand row_demand(const KvArgs &C, const int32_t *src_idx, const int32_t *dst_idx,
                                             const int32_t *n_tokens, int T, int b) {
    Demand d = {-1, 0, 0, false};
    uint32_t bits = 0;
    int np = 0;
    const int dst = dst_idx[b];
    const int src = FORK ? src_idx[b] : dst;
    if (src >= 0 && dst >= 0) {
        const int len = kv_slot_length(C, src, &np, &bits);
        if (len >= 0) {
            if (FORK) {
                if (dst >= C.num_slots) {
                    bits = GDN_SPEC_ST_SLOT_OOR;
                } else if (C.length[dst] != 0 || C.n_pages[dst] != 0) {
                    bits = GDN_SPEC_ST_SLOT_BUSY;
                } else {
                    d = {dst, len >> C.logP, (len & (C.P - 1)) ? 1 : 0, true};
                }
            } else {
                const int n = n_tokens ? n_tokens[b] : T;
                const int64_t want = ((int64_t)len + n + C.P - 1) >> C.logP;
                if (n < 0 || n > T) {
                    bits = GDN_SPEC_ST_ACCEPT_RANGE;
                } else if (want > C.max_pages) {
                    bits = GDN_SPEC_ST_NO_PAGES;
                } else {
                    d = {dst, np, want > np ? (int)want - np : 0, true};
                }
            }
        }
    }
    if (bits) atomicOr(C.status, bits);
    return d;
}

// Word w of the free pages, without bits past the last page (which a caller's
// bitmap may hold: pages of those numbers have no counts to write).
__device__ __forceinline__ uint32_t free_word(const KvArgs &C, int w) {
    const int left = C.num_pages - w * 32;   // w is below 2^26
    if (left <= 0) return 0u;
    const uint32_t bits = C.free_bits[w];
    return left < 32 ? bits & ((1u << left) - 1) : bits;
}

// Whether one of the first n entries of a slot's table, as far as they fall to this
// lane, is no page.
__device__ __forceinline__ bool bad_pages(const KvArgs &C, int slot, int n, int lane, int lanes) {
    const int32_t *t = C.page_table + (int64_t)slot * C.max_pages;
    bool bad = false;
#pragma unroll 4
    for (int i = lane; i < n; i += lanes) bad |= (uint32_t)t[i] >= (uint32_t)C.num_pages;
    return bad;
}

// done[b]: the pages of row b's source are pages, as far as its committed tokens
// reach (other reasons to refuse a row are the allocation's).  A block a row.
__global__ void __launch_bounds__(kCopyThreads) kv_fork_check_kernel(KvArgs C, const int32_t *__restrict__ src_idx,
                                                                     int32_t *__restrict__ done) {
    grid_dep_wait();
    grid_dep_launch();
    const int src = src_idx[blockIdx.x];
    int np;
    uint32_t bits;
    const int len = kv_slot_length(C, src, &np, &bits);
    const bool bad = len > 0 && bad_pages(C, src, (int)(((int64_t)len + C.P - 1) >> C.logP), threadIdx.x, kCopyThreads);
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) done[blockIdx.x] = !any;
}

// Hand out pages for every row (FORK: the page of a partly filled tail, and the
// destination's counts).  Demand sums are held below 2^31 by the host.  A fork's row
// whose source holds an entry that is no page is refused like the others, before it
// asks for any: `checked` says that done[] has the answer, else a warp a row looks
// at the entries here.
template <bool FORK>
__global__ void __launch_bounds__(kAllocThreads) kv_alloc_kernel(KvArgs C, const int32_t *__restrict__ src_idx,
                                                                 const int32_t *__restrict__ dst_idx, int B, int T,
                                                                 const int32_t *__restrict__ n_tokens, bool checked,
                                                                 int32_t *__restrict__ done) {
    __shared__ int warp_sums[33];
    __shared__ int ends[kAllocRows + 1];   // running demand before row b
    __shared__ uint32_t word_s[kAllocThreads];
    __shared__ int rank_s[kAllocThreads];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const int words = (C.num_pages + 31) >> 5;
    const uint32_t first = free_word(C, tid);   // on its way while the rows' chain of loads runs
    bool mine_ok = false;                                         // of row tid
    int total = 0;
    for (int b0 = 0; b0 < B; b0 += kAllocThreads) {
        const int b = b0 + tid;
        Demand d = {-1, 0, 0, false};
        if (b < B) d = row_demand<FORK>(C, src_idx, dst_idx, n_tokens, T, b);
        if (FORK) {
            bool bad = false;
            if (checked) {
                bad = d.ok && !done[b];
            } else {
                word_s[tid] = d.ok ? d.have + d.need : 0;   // entries in use
                rank_s[tid] = d.ok ? src_idx[b] : 0;
                __syncthreads();
                for (int r = tid >> 5; r < min(kAllocThreads, B - b0); r += kAllocThreads >> 5) {
                    const bool lane_bad = bad_pages(C, rank_s[r], word_s[r], tid & 31, 32);
                    if (__any_sync(0xffffffffu, lane_bad) && (tid & 31) == 0) rank_s[r] = -1;
                }
                __syncthreads();
                bad = rank_s[tid] < 0;
            }
            if (bad) {
                atomicOr(C.status, GDN_SPEC_ST_PAGE_OOR);
                d = {-1, 0, 0, false};
            }
        }
        int chunk;
        const int before = block_scan(d.need, warp_sums, &chunk);
        if (b < B) {
            ends[b + 1] = total + before + d.need;
            done[b] = d.ok ? 1 : 0;
            if (b0 == 0) mine_ok = d.ok;
        }
        total += chunk;
    }
    if (tid == 0) ends[0] = 0;
    // free pages, counted only when something is asked for
    int avail = 0;
    if (total > 0) {
        int mine = __popc(first);
        for (int w = tid + kAllocThreads; w < words; w += kAllocThreads) mine += __popc(free_word(C, w));
        block_scan(mine, warp_sums, &avail);
    }
    __syncthreads();
    // Rank r of the free bits goes to the row whose demand spans r.  Rows are served while the running demand
    // (which does not decrease) is available, so the ranks in use are those below `give`.
    int give = total;
    if (total > avail) {
        int lo = 0, hi = B;   // the last row that fits
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ends[mid] <= avail) lo = mid; else hi = mid - 1;
        }
        give = ends[lo];
    }
    int base = 0;
    for (int w0 = 0; w0 < words && base < give; w0 += kAllocThreads) {
        const int w = w0 + tid;
        const uint32_t bits = w0 == 0 ? first : free_word(C, w);
        int chunk;
        const int before = block_scan(__popc(bits), warp_sums, &chunk);   // of the slice's words below
        word_s[tid] = bits;
        rank_s[tid] = before;
        __syncthreads();
        const int take = min(chunk, give - base);
        for (int r = tid; r < take; r += kAllocThreads) {
            int lo = 0, hi = kAllocThreads - 1;   // last word with no more than r before it
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (rank_s[mid] <= r) lo = mid; else hi = mid - 1;
            }
            int k = r - rank_s[lo], bit = 0;      // the word's k-th set bit
            uint32_t x = word_s[lo];
#pragma unroll
            for (int half = 16; half > 0; half >>= 1) {
                const int below = __popc(x & ((1u << half) - 1));
                if (k >= below) {
                    k -= below;
                    x >>= half;
                    bit += half;
                }
            }
            const int page = (w0 + lo) * 32 + bit, rank = base + r;
            lo = 0, hi = B - 1;                   // first row whose running demand exceeds the rank
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (ends[mid + 1] > rank) hi = mid; else lo = mid + 1;
            }
            const int slot = dst_idx[lo];
            const int have = FORK ? (C.length[src_idx[lo]] >> C.logP) : C.n_pages[slot];
            C.page_table[(int64_t)slot * C.max_pages + have + (rank - ends[lo])] = page;
            C.ref[page] = 1;
        }
        // the word's lowest bits are gone
        int mine = min(__popc(bits), max(take - before, 0));
        uint32_t left = bits;
        if (mine == __popc(bits)) left = 0;
        else
            for (; mine > 0; --mine) left &= left - 1;
        if (left != bits) C.free_bits[w] = left;
        base += chunk;
        __syncthreads();   // the slice's words were read
    }
    __syncthreads();   // the counts were read above
    for (int b = tid; b < B; b += kAllocThreads) {
        if (b == tid ? !mine_ok : !done[b]) continue;
        const int need = ends[b + 1] - ends[b];
        if (need > 0 && ends[b + 1] > give) {
            done[b] = 0;
            atomicOr(C.status, GDN_SPEC_ST_NO_PAGES);
            continue;
        }
        const int slot = dst_idx[b];
        if (FORK) {
            const int len = C.length[src_idx[b]];
            C.n_pages[slot] = (len >> C.logP) + need;
            C.length[slot] = len;
        } else if (need > 0) {
            C.n_pages[slot] += need;
        }
    }
}

// The rest of a fork: shared pages, and the copied rows of the last page.  The entries
// are pages, unless a destination is also a source, which the call forbids: the
// tests here keep that inside the pool too.
// Grid (rows, parts): a block copies the rows of one head of one layer's keys or
// values at a time (one contiguous run), four 16-byte loads in flight per thread.
__global__ void __launch_bounds__(kCopyThreads) kv_fork_copy_kernel(KvArgs C, const int32_t *__restrict__ src_idx,
                                                                    const int32_t *__restrict__ dst_idx,
                                                                    const int32_t *done, int es) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.x, tid = threadIdx.x;
    if (!done[b]) return;
    const int src = src_idx[b], dst = dst_idx[b];
    const int len = C.length[src], full = len >> C.logP, part = len & (C.P - 1);
    const int32_t *st = C.page_table + (int64_t)src * C.max_pages;
    int32_t *dt = C.page_table + (int64_t)dst * C.max_pages;
    for (int i = blockIdx.y * kCopyThreads + tid; i < full; i += gridDim.y * kCopyThreads) {
        const int page = st[i];
        if (page >= 0 && page < C.num_pages) atomicAdd(&C.ref[page], 1);
        else atomicOr(C.status, GDN_SPEC_ST_PAGE_OOR);
        dt[i] = page;
    }
    if (part == 0) return;
    const int from = st[full], to = dt[full];
    if (from < 0 || from >= C.num_pages || to < 0 || to >= C.num_pages) {
        if (tid == 0) atomicOr(C.status, GDN_SPEC_ST_PAGE_OOR);
        return;
    }
    const int64_t page_bytes = (int64_t)C.P * C.D * es;
    const int run = part * C.D * es / 16;   // 16-byte pieces of one head's rows
    const int units = C.n_layers * C.HKV * 2;
    for (int u = blockIdx.y; u < units; u += gridDim.y) {
        const int which = u & 1, lh = u >> 1, layer = lh / C.HKV, h = lh - layer * C.HKV;
        char *pool = static_cast<char *>(which ? C.v : C.k);
        const int4 *s = reinterpret_cast<const int4 *>(
            pool + (((int64_t)layer * C.num_pages + from) * C.HKV + h) * page_bytes);
        int4 *d = reinterpret_cast<int4 *>(pool + (((int64_t)layer * C.num_pages + to) * C.HKV + h) * page_bytes);
        int i = tid;
        for (; i + 3 * kCopyThreads < run; i += 4 * kCopyThreads) {
            int4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = s[i + j * kCopyThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i + j * kCopyThreads] = x[j];
        }
        for (; i < run; i += kCopyThreads) d[i] = s[i];
    }
}

// A commit's row, decided by one warp: the committed length, or -1 (nothing is
// done).  Every lane returns the same.
__device__ __forceinline__ int commit_row(const KvArgs &C, int slot, int acc, int T, const int32_t *path, int lane,
                                          uint32_t *bits) {
    *bits = 0;
    if (slot < 0) return -1;
    int reach = acc;   // drafts up to the last accepted one
    if (path) {
        bool fine = acc >= 0 && acc <= T;
        if (fine && acc > 0) {
            const int last = path[acc - 1];
            fine = last >= 0 && last < T;
            reach = last + 1;
        }
        if (fine)
            for (int i = lane; i < acc; i += 32) {
                const int p = path[i], before = i ? path[i - 1] : -1;
                if (p <= before) fine = false;
            }
        if (!__all_sync(0xffffffffu, fine)) { *bits = GDN_SPEC_ST_ACCEPT_RANGE; return -1; }
    }
    const int len = kv_row(C, slot, reach, T, bits);
    if (len < 0) return -1;
    bool pages = true;
    if (path)
        for (int i = lane; i < acc; i += 32)
            if (kv_token_row(C, slot, len + path[i]) < 0 || kv_token_row(C, slot, len + i) < 0) pages = false;
    if (!__all_sync(0xffffffffu, pages)) { *bits = GDN_SPEC_ST_PAGE_OOR; return -1; }
    return len;
}

// Accepted drafts move together.  A thread owns one 16-byte column of one head
// of one layer's keys or values and walks the path upwards, eight loads before
// their eight stores.  In place this is safe: a path ascends, so path[i] >= i, and
// the rows written so far, all below i, are never the source of a later move.
// Leading nodes with path[i] == i stay.  ADVANCE: the launch has one block per row,
// which moves the length as well once it has read it.
template <bool ADVANCE>
__global__ void __launch_bounds__(kCopyThreads) kv_move_kernel(KvArgs C, const int32_t *__restrict__ slot_idx, int T,
                                                               const int32_t *__restrict__ path,
                                                               const int32_t *__restrict__ accept_len, int es) {
    __shared__ int from_s[kMoveMaxT], to_s[kMoveMaxT];
    __shared__ int n_s;
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int slot = slot_idx[b], acc = accept_len[b];
    const int32_t *p = path + (int64_t)b * T;
    if (tid < 32) {
        uint32_t bits;
        const int len = commit_row(C, slot, acc, T, p, tid, &bits);
        if (tid == 0 && bits && blockIdx.y == 0) atomicOr(C.status, bits);
        // a path that ascends leaves its first nodes where they are and moves all others
        int stay = 0, n = 0;
        if (len >= 0) {
            for (int i0 = 0; i0 < acc; i0 += 32) stay += __popc(__ballot_sync(0xffffffffu, i0 + tid < acc && p[i0 + tid] == i0 + tid));
            n = acc - stay;
            for (int i = tid; i < n; i += 32) {
                from_s[i] = (int)kv_token_row(C, slot, len + p[stay + i]);
                to_s[i] = (int)kv_token_row(C, slot, len + stay + i);
            }
        }
        if (tid == 0) {
            n_s = n;
            if (ADVANCE && len >= 0 && acc > 0) C.length[slot] = len + acc;
        }
    }
    __syncthreads();
    const int n = n_s;
    if (n == 0) return;
    const int cols = C.D * es / 16, units = C.n_layers * C.HKV * 2 * cols;
    const int64_t head_pieces = (int64_t)C.P * cols;
    for (int u = blockIdx.y * kCopyThreads + tid; u < units; u += gridDim.y * kCopyThreads) {
        const int lh2 = u / cols, col = u - lh2 * cols, which = lh2 & 1, lh = lh2 >> 1;
        const int layer = lh / C.HKV, h = lh - layer * C.HKV;
        int4 *pool = reinterpret_cast<int4 *>(which ? C.v : C.k) + col;
        const auto at = [&](int row) {
            return (((int64_t)layer * C.num_pages + (row >> C.logP)) * C.HKV + h) * head_pieces +
                   (int64_t)(row & (C.P - 1)) * cols;
        };
        int i = 0;
        for (; i + 8 <= n; i += 8) {
            int4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = pool[at(from_s[i + j])];
#pragma unroll
            for (int j = 0; j < 8; ++j) pool[at(to_s[i + j])] = x[j];
        }
        for (; i < n; ++i) pool[at(to_s[i])] = pool[at(from_s[i])];
    }
}

// length += accept_len for the rows that the move took, one warp a row.
__global__ void kv_advance_kernel(KvArgs C, const int32_t *__restrict__ slot_idx, int B, int T,
                                  const int32_t *__restrict__ path, const int32_t *__restrict__ accept_len) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (b >= B) return;
    const int slot = slot_idx[b], acc = accept_len[b];
    uint32_t bits;
    const int len = commit_row(C, slot, acc, T, path ? path + (int64_t)b * T : nullptr, lane, &bits);
    if (lane == 0) {
        if (bits) atomicOr(C.status, bits);
        if (len >= 0 && acc > 0) C.length[slot] = len + acc;
    }
}

// One block per row: the slot's pages lose a holder, and become free at zero.
__global__ void __launch_bounds__(kCopyThreads) kv_free_kernel(KvArgs C, const int32_t *__restrict__ slot_idx) {
    grid_dep_wait();
    grid_dep_launch();
    const int slot = slot_idx[blockIdx.x], tid = threadIdx.x;
    int np;
    uint32_t bits;
    const int len = kv_slot_length(C, slot, &np, &bits);
    if (len < 0) {
        if (tid == 0 && bits) atomicOr(C.status, bits);
        return;
    }
    int32_t *t = C.page_table + (int64_t)slot * C.max_pages;
    for (int i = tid; i < np; i += kCopyThreads) {
        const int page = t[i];
        t[i] = -1;
        if (page < 0 || page >= C.num_pages) {
            atomicOr(C.status, GDN_SPEC_ST_PAGE_OOR);
            continue;
        }
        const int before = atomicSub(&C.ref[page], 1);
        if (before == 1) {
            atomicOr(&C.free_bits[page >> 5], 1u << (page & 31));
        } else if (before <= 0) {   // nobody held it: the counts are not a cache's
            atomicAdd(&C.ref[page], 1);
            atomicOr(C.status, GDN_SPEC_ST_CURSOR_CORRUPT);
        }
    }
    __syncthreads();   // every thread has read the counts
    if (tid == 0) {
        C.n_pages[slot] = 0;
        C.length[slot] = 0;
    }
}

__global__ void __launch_bounds__(kCopyThreads) kv_init_kernel(KvArgs C) {
    const int64_t i0 = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x, step = (int64_t)gridDim.x * kCopyThreads;
    const int64_t entries = (int64_t)C.num_slots * C.max_pages;
    for (int64_t i = i0; i < entries; i += step) C.page_table[i] = -1;
    for (int64_t i = i0; i < C.num_slots; i += step) C.n_pages[i] = C.length[i] = 0;
    for (int64_t i = i0; i < C.num_pages; i += step) C.ref[i] = 0;
    const int words = (C.num_pages + 31) >> 5, rest = C.num_pages & 31;
    for (int64_t i = i0; i < words; i += step) C.free_bits[i] = (i == words - 1 && rest) ? (1u << rest) - 1 : 0xffffffffu;
}

cudaError_t launch_kv_init(const KvArgs &C, cudaStream_t stream) {
    kv_init_kernel<<<256, kCopyThreads, 0, stream>>>(C);
    return cudaGetLastError();
}

int kv_alloc_max_rows() { return kAllocRows; }
int kv_move_max_window() { return kMoveMaxT; }

cudaError_t launch_kv_reserve(const KvArgs &C, const int32_t *slot_idx, int B, int T, const int32_t *n_tokens,
                              int32_t *done, cudaStream_t stream) {
    return launch_dependent(kv_alloc_kernel<false>, dim3(1), dim3(kAllocThreads), 0, stream, C, slot_idx, slot_idx, B,
                            T, n_tokens, false, done);
}

// Blocks along a row's layers, heads, keys and values: as many as there are
// runs, but no more than `blocks` in all.
static int copy_parts(int B, int most, int blocks) {
    const int want = (blocks + B - 1) / B;
    return most < want ? (most < 1 ? 1 : most) : want;
}

cudaError_t launch_kv_fork(const KvArgs &C, const int32_t *src_idx, const int32_t *dst_idx, int B, int32_t *done,
                           int es, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const bool check = (int64_t)B * C.max_pages > kForkInline;
    if (check) e = launch_dependent(kv_fork_check_kernel, dim3(B), dim3(kCopyThreads), 0, stream, C, src_idx, done);
    if (e == cudaSuccess)
        e = launch_dependent(kv_alloc_kernel<true>, dim3(1), dim3(kAllocThreads), 0, stream, C, src_idx, dst_idx, B, 0,
                             (const int32_t *)nullptr, check, done);
    if (e != cudaSuccess) return e;
    const int parts = copy_parts(B, C.n_layers * C.HKV * 2, 8192);
    return launch_dependent(kv_fork_copy_kernel, dim3(B, parts), dim3(kCopyThreads), 0, stream, C, src_idx, dst_idx,
                            (const int32_t *)done, es);
}

cudaError_t launch_kv_commit(const KvArgs &C, const int32_t *slot_idx, int B, int T, const int32_t *path,
                             const int32_t *accept_len, int es, cudaStream_t stream) {
    if (path) {
        const int64_t units = (int64_t)C.n_layers * C.HKV * 2 * (C.D * es / 16);
        const int64_t need = (units + kCopyThreads - 1) / kCopyThreads;
        // one block per row saves the second launch (some 2 us) where a thread then walks no more than four columns
        if (need <= 4)
            return launch_dependent(kv_move_kernel<true>, dim3(B, 1), dim3(kCopyThreads), 0, stream, C, slot_idx, T, path,
                                    accept_len, es);
        // some eight blocks an SM: each starts with a chain of loads (slot, counts, path, pages)
        const int parts = copy_parts(B, need > 1280 ? 1280 : (int)need, 1280);
        cudaError_t e = launch_dependent(kv_move_kernel<false>, dim3(B, parts), dim3(kCopyThreads), 0, stream, C, slot_idx, T,
                                         path, accept_len, es);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kv_advance_kernel, dim3((B + 3) / 4), dim3(128), 0, stream, C, slot_idx, B, T, path,
                            accept_len);
}

cudaError_t launch_kv_free(const KvArgs &C, const int32_t *slot_idx, int B, cudaStream_t stream) {
    return launch_dependent(kv_free_kernel, dim3(B), dim3(kCopyThreads), 0, stream, C, slot_idx);
}

}  // namespace gdnspec
