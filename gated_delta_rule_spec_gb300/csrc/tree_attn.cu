// tree_attn.cu -- attention of a window of drafted tokens over the paged cache on
// the CUDA cores (fp32, and groups of more than 128 heads), and the join of split
// items for both kernels.
//
// Per query row, one pass over the keys with a running maximum m and sum l in
// powers of two: for a tile's scores s (times scale log2 e),
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v,
// and the row's output is o / l.  A row that has seen nothing yet has m = -inf, l = 0.
//
// A block holds MT query rows and walks tiles of 32 keys, copied asynchronously into
// one of two buffers while the other is worked on.  Four warps share a tile, eight
// keys each, and from 16 rows on two such fours halve the rows: every warp keeps
// a running maximum and sum of its own for its rows and keys, and the four are
// merged in shared memory at the end of a piece.  So a key or value is read from
// shared memory by one or two warps only.  Of a warp's scores lane (g, k) forms rows
// g, g + 4, ... with key k; the maximum is a shuffle over eight lanes, and the sums
// run over output columns, VEC consecutive ones per lane.  Rows of keys and queries
// are padded by 16 bytes, so that the pieces read together fall in different banks.
// 16 sequences of 5000 tokens, 4 heads of 128 fp32, 8 drafts: 73 us, 3.4 TB/s, half of
// HBM's rate, with the issue slots 58% and the shared-memory pipe 53% busy: no pipe
// bounds it, the latency of tiles between two block barriers each does.  8 of them with
// 32 rows a head: 87 us, where a warp's 16 multiply-adds for 5 wide reads take 8.7
// wavefronts; the pipe is busy 58% of the kernel and the issue slots 57%.
#include "attn_common.cuh"
#include "launch_setup.cuh"

namespace gdnspec {

constexpr int kAttnTile = 32;     // keys of a tile
constexpr int kSplit = 4;         // warps that share a tile
constexpr int kWarpKeys = kAttnTile / kSplit;

// Bytes at the front: the two buffers of keys and values, and at a piece's end the four warps' sums in their place.
__host__ __device__ constexpr size_t attn_front_bytes(int D, int MT, int es) {
    const size_t tiles = (size_t)2 * kAttnTile * (2 * D * es + 16), sums = (size_t)kSplit * MT * (D + 4) * sizeof(float);
    return tiles > sums ? tiles : sums;
}

size_t tree_attn_smem(int D, int MT, int es) {   // and queries, probabilities, (maximum, sum)
    return attn_front_bytes(D, MT, es) + (size_t)MT * (D * es + 16) + sizeof(float) * (size_t)kSplit * MT * (kWarpKeys + 2);
}

// (m, l, o) of a row's four dims, as (maximum in log2 units, sum, unnormalised sums)
struct JoinSum {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 ml, float4 po) {
        if (ml.y == 0.0f) return;   // that piece saw nothing, its sums may be anything
        const float mn = fmaxf(m, ml.x), wa = exp2f(m - mn), wb = exp2f(ml.x - mn);
        l = l * wa + ml.y * wb;
        o.x = o.x * wa + po.x * wb;
        o.y = o.y * wa + po.y * wb;
        o.z = o.z * wa + po.z * wb;
        o.w = o.w * wa + po.w * wb;
        m = mn;
    }
};

template <typename IO>
__device__ __forceinline__ void join_put(const AttnArgs &A, const JoinSum &j, int64_t row, int d4) {
    const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l;
    IO out[4] = {from_f32<IO>(j.o.x * inv), from_f32<IO>(j.o.y * inv), from_f32<IO>(j.o.z * inv), from_f32<IO>(j.o.w * inv)};
    IO *op = static_cast<IO *>(A.out) + row * A.C.D + 4 * d4;
    if (sizeof(IO) == 2) *reinterpret_cast<uint2 *>(op) = *reinterpret_cast<const uint2 *>(out);
    else *reinterpret_cast<uint4 *>(op) = *reinterpret_cast<const uint4 *>(out);
    if (A.lse && d4 == 0) A.lse[row] = attn_lse(j.m, j.l);
}

template <typename IO> __device__ __forceinline__ float4 load4(const IO *p);
template <> __device__ __forceinline__ float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}
template <typename IO> __device__ __forceinline__ float2 load2(const IO *p);
template <> __device__ __forceinline__ float2 load2<float>(const float *p) { return *reinterpret_cast<const float2 *>(p); }
template <> __device__ __forceinline__ float2 load2<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}

__device__ __forceinline__ uint32_t smem_of(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Sixteen bytes from global to shared memory; zeros where !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

// Blocks of an SM that the registers leave room for.  (At the 128 registers of two blocks
// the kernels of 24 and 32 rows keep 4 to 92 bytes a thread in local memory, most of
// them with 32 rows of 128 fp32.)
__host__ __device__ constexpr int attn_blocks(int WR, int RW, int NG) {
    return WR == 2 ? (NG == 2 ? 1 : 2) : NG == 2 ? 2 : 4;
}

// acc += p v over a warp's keys; TEST: a probability of zero takes nothing from its value.
template <typename IO, int RW, int VEC, int NG, bool TEST>
__device__ __forceinline__ void add_values(float (&acc)[RW][NG * VEC], const float *p_s, const IO *v_s, int D, int lane) {
#pragma unroll 1
    for (int k = 0; k < kWarpKeys; k += 4) {
        float v[4][NG * VEC];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int d = (g * 32 + lane) * VEC;
                if (VEC == 4) {
                    const float4 x = d < D ? load4<IO>(v_s + (k + e) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[e][g * VEC] = x.x, v[e][g * VEC + 1] = x.y, v[e][g * VEC + 2] = x.z, v[e][g * VEC + 3] = x.w;
                } else {
                    const float2 x = d < D ? load2<IO>(v_s + (k + e) * D + d) : make_float2(0.f, 0.f);
                    v[e][g * VEC] = x.x, v[e][g * VEC + 1] = x.y;
                }
            }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const float4 p = *reinterpret_cast<const float4 *>(p_s + r * kWarpKeys + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = e == 0 ? p.x : e == 1 ? p.y : e == 2 ? p.z : p.w;
                if (!TEST || x != 0.0f) {
#pragma unroll
                    for (int j = 0; j < NG * VEC; ++j) acc[r][j] = fmaf(x, v[e][j], acc[r][j]);
                }
            }
        }
    }
}

// WR fours of warps with RW rows each (MT = WR RW); NG groups of 32 VEC output columns.
template <typename IO, int WR, int RW, int VEC, int NG>
__global__ void __launch_bounds__(32 * kSplit * WR, attn_blocks(WR, RW, NG)) tree_attn_kernel(const __grid_constant__ AttnArgs A) {
    constexpr int kThreads = 32 * kSplit * WR, MT = WR * RW, R = RW / 4;
    constexpr int kPiece = 16 / sizeof(IO);                                     // elements of 16 bytes
    constexpr int kCopied = kAttnTile * 32 / kThreads;                          // tokens that a warp copies
    constexpr int kRun = NG * 32 * VEC / kPiece, kLanes = kRun < 32 ? kRun : 32;   // pieces of a token, lanes that copy it
    constexpr int kSteps = kRun / kLanes;
    constexpr int kChains = R == 1 ? 4 : R == 2 ? 2 : 1;   // sums of a score, so that their additions overlap
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scratch[kAttnScratch];
    const int D = A.C.D, D4 = D >> 2, KLD = D + kPiece, QLD = D + 4;
    IO *const Ks = reinterpret_cast<IO *>(smem);                              // [2][32][D + 16 bytes]
    IO *const Vs = Ks + 2 * kAttnTile * KLD;                                  // [2][32][D]
    float *const Os = reinterpret_cast<float *>(smem);                        // [4][MT][D + 4], at a piece's end
    IO *const Qs = reinterpret_cast<IO *>(smem + attn_front_bytes(D, MT, sizeof(IO)));   // [MT][D + 16 bytes]
    float *const Ps = reinterpret_cast<float *>(Qs + MT * KLD);                                          // [warps][RW][8]
    float2 *const MLs = reinterpret_cast<float2 *>(Ps + kSplit * MT * kWarpKeys);   // [4][MT]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wk = warp % kSplit, r0 = warp / kSplit * RW;   // the warp's keys and first row
    const int kl = lane & 7, rg = lane >> 3;                 // the lane's key and first row of them
    const int group = blockIdx.x / A.NQT, qt = blockIdx.x - group * A.NQT;
    float *const my_p = Ps + warp * RW * kWarpKeys;
    const IO *const my_q = Qs + (r0 + rg) * KLD;
    const int at = lane % kLanes * kPiece;                   // the lane's element of the tokens that it copies
    const uint32_t k_dst = smem_of(Ks + (warp * kCopied + lane / kLanes) * KLD + at);
    const uint32_t v_dst = smem_of(Vs + (warp * kCopied + lane / kLanes) * D + at);
    grid_dep_wait();

    attn_dead_rows<IO>(A, blockIdx.x, gridDim.x, tid, kThreads);
    const AttnPlan plan = attn_plan<kThreads>(A, group, blockIdx.x == 0, scratch);
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    bool any = walk.next(A, &pc);
    if (tid == 0 && qt == 0) attn_note(A, group, any, pc, plan.chunk);
    for (; any; any = walk.next(A, &pc)) {
        const int live = min(MT, pc.cnt * A.G - qt * MT);   // rows of this query tile
        if (live <= 0) continue;
        const int kv = pc.len + pc.cnt, pieces = D / kPiece;
        const int fr = warp * kCopied + lane % kCopied;   // this lane looks up that token of a tile
        const bool together = A.C.P >= kAttnTile;
        const auto page_of = [&](int t) {   // of this thread's token of tile t
            const int tok = t * kAttnTile + fr;
            return t < pc.t1 && tok < kv ? A.C.page_table[(int64_t)pc.slot * A.C.max_pages + (tok >> A.C.logP)] : 0;
        };
        const auto fetch = [&](int t, int buf, int page) {
            const int tok = t * kAttnTile + fr;
            const bool ok = page >= 0 && page < A.C.num_pages, there = tok < kv && ok;
            if (tok < kv && !ok) atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
            const int64_t mine = there ? kv_elem(A.C, A.layer, pc.h, ((int64_t)page << A.C.logP) + (tok & (A.C.P - 1))) : -1;
            // Rows past the end are zeros, whatever the page holds there.  Where a page holds a tile its rows follow the
            // warp's first one.
            const int64_t start = together ? __shfl_sync(0xffffffffu, mine, 0) : 0;
            const int left = kv - t * kAttnTile - warp * kCopied;
            const uint32_t kd = k_dst + buf * kAttnTile * KLD * (uint32_t)sizeof(IO);
            const uint32_t vd = v_dst + buf * kAttnTile * D * (uint32_t)sizeof(IO);
#pragma unroll
            for (int i = 0; i < kCopied; i += 32 / kLanes) {
                const int r = i + lane / kLanes;
                int64_t e = together ? (r < left ? start : -1) : __shfl_sync(0xffffffffu, mine, r);
                const bool live_row = e >= 0;
                if (together) e = max(start, (int64_t)0) + r * D;
                else if (!live_row) e = 0;
                const IO *k = static_cast<const IO *>(A.C.k) + e + at, *v = static_cast<const IO *>(A.C.v) + e + at;
#pragma unroll
                for (int c = 0; c < kSteps; ++c) {
                    if (at + c * kLanes * kPiece >= D) break;
                    copy16(kd + (i * KLD + c * kLanes * kPiece) * (uint32_t)sizeof(IO), k + c * kLanes * kPiece, live_row);
                    copy16(vd + (i * D + c * kLanes * kPiece) * (uint32_t)sizeof(IO), v + c * kLanes * kPiece, live_row);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int page = page_of(pc.t0);
        __syncthreads();   // the piece before is done with shared memory
        for (int r = warp * (32 / kLanes) + lane / kLanes; r < MT; r += kThreads / kLanes) {
            const IO *q = static_cast<const IO *>(A.q) + (r < live ? attn_out_row(A, pc.b, pc.h, qt * MT + r) * D : 0);
            for (int c = lane % kLanes; c < pieces; c += kLanes) copy16(smem_of(Qs + r * KLD + c * kPiece), q + c * kPiece, r < live);
        }
        fetch(pc.t0, 0, page);
        page = page_of(pc.t0 + 1);   // always a tile ahead of its copy
        uint64_t mask[R];
        float m[R], l[R];   // of the warp's keys; l: this lane's only, until the end
        float acc[RW][NG * VEC] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = r0 + rg + 4 * i;
            mask[i] = r < live ? attn_mask(A, pc.b, (qt * MT + r) / A.G) : 0;
            m[i] = -INFINITY;
            l[i] = 0.0f;
        }
        for (int t = pc.t0; t < pc.t1; ++t) {
            const int buf = (t - pc.t0) & 1, k0 = t * kAttnTile + wk * kWarpKeys;
            if (t + 1 < pc.t1) {
                fetch(t + 1, buf ^ 1, page);
                page = page_of(t + 2);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            const IO *kp = Ks + (buf * kAttnTile + wk * kWarpKeys + kl) * KLD;
            const IO *vp = Vs + (buf * kAttnTile + wk * kWarpKeys) * D;
            float s[R][kChains] = {};
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                const float4 kx = load4<IO>(kp + d);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float4 qx = load4<IO>(my_q + i * 4 * KLD + d);
                    s[i][0] = fmaf(qx.x, kx.x, s[i][0]);
                    s[i][1 % kChains] = fmaf(qx.y, kx.y, s[i][1 % kChains]);
                    s[i][2 % kChains] = fmaf(qx.z, kx.z, s[i][2 % kChains]);
                    s[i][3 % kChains] = fmaf(qx.w, kx.w, s[i][3 % kChains]);
                }
            }
            const int node = k0 + kl - pc.len;   // < 0: committed
            const bool drafts = k0 + kWarpKeys > pc.len;
            float al[R];
            bool up = false;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float x = kChains == 4 ? (s[i][0] + s[i][1 % kChains]) + (s[i][2 % kChains] + s[i][3 % kChains])
                          : kChains == 2 ? s[i][0] + s[i][1 % kChains] : s[i][0];
                x *= A.scale_log2;
                if (drafts && !(k0 + kl < kv && (node < 0 || ((mask[i] >> node) & 1)))) x = -INFINITY;
                float top = x;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float mn = fmaxf(m[i], top), base = mn == -INFINITY ? 0.0f : mn;
                const float p = exp2f(x - base);
                al[i] = exp2f(m[i] - base);
                up |= mn > m[i];
                m[i] = mn;
                l[i] = l[i] * al[i] + p;
                my_p[(rg + 4 * i) * kWarpKeys + kl] = p;
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    const float a = __shfl_sync(0xffffffffu, al[r / 4], (r & 3) * 8);
#pragma unroll
                    for (int j = 0; j < NG * VEC; ++j) acc[r][j] *= a;
                }
            }
            __syncwarp();
            // Keys that hold drafted tokens leave masked ones out by a test, so that an infinity or NaN there stays
            // without effect; committed tokens are seen by every row.
            if (drafts) add_values<IO, RW, VEC, NG, true>(acc, my_p, vp, D, lane);
            else add_values<IO, RW, VEC, NG, false>(acc, my_p, vp, D, lane);
            __syncthreads();   // the buffer may be filled again
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if (kl == 0) MLs[wk * MT + r0 + rg + 4 * i] = make_float2(m[i], l[i]);
        }
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int d = (g * 32 + lane) * VEC;
                float *o = Os + (wk * MT + r0 + r) * QLD + d;
                if (d >= D) continue;
                if (VEC == 4) *reinterpret_cast<float4 *>(o) = make_float4(acc[r][g * VEC], acc[r][g * VEC + 1], acc[r][g * VEC + 2], acc[r][g * VEC + 3]);
                else *reinterpret_cast<float2 *>(o) = make_float2(acc[r][g * VEC], acc[r][g * VEC + 1]);
            }
        __syncthreads();
        const int64_t part = (int64_t)blockIdx.x * 2 + pc.side;
        for (int x = tid; x < MT * D4; x += kThreads) {
            // in the order of where it goes: along a row of the output, or along the rows of a piece
            const int r = pc.whole() ? x / D4 : x % MT, d4 = pc.whole() ? x - r * D4 : x / MT;
            if (r >= live) continue;
            JoinSum sum;
#pragma unroll
            for (int w = 0; w < kSplit; ++w) sum.add(MLs[w * MT + r], *reinterpret_cast<const float4 *>(Os + (w * MT + r) * QLD + 4 * d4));
            if (pc.whole()) {
                join_put<IO>(A, sum, attn_out_row(A, pc.b, pc.h, qt * MT + r), d4);
            } else {
                A.part_o[(part * D4 + d4) * MT + r] = sum.o;
                if (d4 == 0) A.part_ml[part * MT + r] = make_float2(sum.m, sum.l);
            }
        }
    }
    grid_dep_launch();
}

// ------------------------------------------------------------------ join

constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = 8;      // threads that share an element's pieces when they are many
constexpr int kJoinMany = 16;      // from so many pieces on

// Block (g, query tile, part), for the item that chunk g starts inside of.  The blocks of all chunks that do share the
// item's elements, so an item of many pieces has as many more blocks (3 rows of 7698 tokens, 28 rows of 256 fp32 each:
// 107 us where the first of them took all, 36 so).  A thread takes the same four dims of one row from every piece, all
// loads of two pieces in flight before they are merged; where an item has many pieces eight threads share an
// element.  Everything about the item is in the chunk's note, so a block starts with one load.
template <typename IO>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs A) {
    __shared__ float4 o_s[kJoinLanes][32];
    __shared__ float2 ml_s[kJoinLanes][32];
    grid_dep_wait();
    const int g = blockIdx.x + 1, qt = blockIdx.y, tid = threadIdx.x, lane = tid & 31, pl = tid >> 5;
    const AttnCut cut = A.cuts[g];
    const int64_t s = (int64_t)g * cut.chunk - cut.t;   // the place of the item's first tile
    if (cut.b < 0 || cut.t == 0) return;   // a cut between items
    const int first = (int)(s / cut.chunk);
    const int live = min(A.MT, cut.cnt * A.G - qt * A.MT);
    if (live <= 0) return;
    const int last = (int)((s + cut.tiles - 1) / cut.chunk);
    const int D4 = A.C.D >> 2, work = live * D4;
    const int block = (g - 1 - first) * gridDim.z + blockIdx.z, blocks = (last - first) * gridDim.z;   // of the item
    const auto part_of = [&](int c) { return ((int64_t)c * A.NQT + qt) * 2 + (c == first ? 1 : 0); };
    if (last - first + 1 < kJoinMany) {
        for (int x = block * kJoinThreads + tid; x < work; x += blocks * kJoinThreads) {
            const int d4 = x / live, r = x - d4 * live;
            JoinSum sum;
            for (int c = first; c <= last; c += 2) {
                const int64_t p0 = part_of(c), p1 = part_of(min(c + 1, last));
                const float2 ml0 = A.part_ml[p0 * A.MT + r], ml1 = A.part_ml[p1 * A.MT + r];
                const float4 o0 = A.part_o[(p0 * D4 + d4) * A.MT + r], o1 = A.part_o[(p1 * D4 + d4) * A.MT + r];
                sum.add(ml0, o0);
                if (c < last) sum.add(ml1, o1);
            }
            join_put<IO>(A, sum, attn_out_row(A, cut.b, cut.h, qt * A.MT + r), d4);
        }
        return;
    }
    for (int x0 = block * 32; x0 < work; x0 += blocks * 32) {
        const int x = x0 + lane, d4 = x / live, r = x - d4 * live;
        JoinSum sum;
        if (x < work)
            for (int c = first + pl; c <= last; c += 4 * kJoinLanes) {   // four pieces' loads in flight
                float2 ml[4];
                float4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int64_t part = part_of(min(c + k * kJoinLanes, last));
                    ml[k] = A.part_ml[part * A.MT + r];
                    o[k] = A.part_o[(part * D4 + d4) * A.MT + r];
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k * kJoinLanes <= last) sum.add(ml[k], o[k]);
            }
        o_s[pl][lane] = sum.o;
        ml_s[pl][lane] = make_float2(sum.m, sum.l);
        __syncthreads();
        if (pl == 0 && x < work) {
#pragma unroll
            for (int w = 1; w < kJoinLanes; ++w) sum.add(ml_s[w][lane], o_s[w][lane]);
            join_put<IO>(A, sum, attn_out_row(A, cut.b, cut.h, qt * A.MT + r), d4);
        }
        __syncthreads();
    }
}

cudaError_t launch_attn_join(const AttnArgs &A, bool bf16, cudaStream_t stream) {
    if (A.groups < 2) return cudaSuccess;
    const int rows = A.T * A.G < A.MT ? A.T * A.G : A.MT;
    int parts = (rows * (A.C.D / 4) + 2 * kJoinThreads - 1) / (2 * kJoinThreads);   // two elements a thread
    if (parts < 4) parts = 4;
    if (parts > 16) parts = 16;
    const dim3 grid(A.groups - 1, A.NQT, parts);
    return bf16 ? launch_dependent(attn_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, stream, A)
                : launch_dependent(attn_join_kernel<float>, grid, dim3(kJoinThreads), 0, stream, A);
}

// ------------------------------------------------------------------ launch

// Rows of a block's query tile: the fewest of 4, 8, 12, 16, 24 and 32 that hold the window; longer windows take tiles of
// 32, or two of 24 (against the next larger tile, geometric means of fp32 shapes: 12 rows 33.7 and 41.1 us, 24 rows
// 34.3 and 40.0 us).  From 16 rows on there are two fours of warps: with one of sixteen rows a warp, 8 sequences of 5000
// tokens, 4 shared heads of 128 fp32, 8 drafts x 2 heads were 80 us against 66.
static int tile_rows(int R) {
    return R <= 4 ? 4 : R <= 8 ? 8 : R <= 12 ? 12 : R <= 16 ? 16 : R <= 24 || (R > 32 && R <= 48) ? 24 : 32;
}
static constexpr int fours(int MT) { return MT <= 12 ? 1 : 2; }

template <typename IO, int MT, int VEC, int NG>
static cudaError_t run_tree_attn(const AttnArgs &A, cudaStream_t st) {
    constexpr int WR = fours(MT);
    static KernelSetup setup;
    const size_t smem = tree_attn_smem(A.C.D, MT, sizeof(IO));
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)tree_attn_kernel<IO, WR, MT / WR, VEC, NG>, smem, &sms);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_attn_kernel<IO, WR, MT / WR, VEC, NG>, dim3(A.groups * A.NQT), dim3(32 * kSplit * WR), smem, st, A);
}

template <typename IO, int MT>
static cudaError_t run_cols(const AttnArgs &A, cudaStream_t st) {
    if (A.C.D <= 64) return run_tree_attn<IO, MT, 2, 1>(A, st);
    if (A.C.D <= 128) return run_tree_attn<IO, MT, 4, 1>(A, st);
    return run_tree_attn<IO, MT, 4, 2>(A, st);
}

template <typename IO>
static cudaError_t run_rows(const AttnArgs &A, cudaStream_t st) {
    switch (A.MT) {
        case 4: return run_cols<IO, 4>(A, st);
        case 8: return run_cols<IO, 8>(A, st);
        case 12: return run_cols<IO, 12>(A, st);
        case 16: return run_cols<IO, 16>(A, st);
        case 24: return run_cols<IO, 24>(A, st);
        default: return run_cols<IO, 32>(A, st);
    }
}

// The cut of the work on a machine of `sms` SMs (MT, TN, NQT, groups).
void tree_attn_cut(AttnArgs *A, int sms, int es) {
    const int R = A->T * A->G;
    A->TN = kAttnTile;
    A->MT = tile_rows(R);
    A->NQT = (R + A->MT - 1) / A->MT;
    const int fit = (int)((size_t)(227 * 1024) / (tree_attn_smem(A->C.D, A->MT, es) + 2048));
    const int most = attn_blocks(fours(A->MT), A->MT / fours(A->MT), A->C.D > 128 ? 2 : 1);
    const int per_sm = fit < 1 ? 1 : fit < most ? fit : most;
    const int groups = sms * per_sm / A->NQT;
    A->groups = groups < 1 ? 1 : groups;
    A->min_chunk = 2;
    A->gap = 1;   // an item's queries, merge and way out take about as long as a tile
}

cudaError_t launch_tree_attn(const AttnArgs &A, bool bf16, cudaStream_t st) {
    const cudaError_t e = bf16 ? run_rows<__nv_bfloat16>(A, st) : run_rows<float>(A, st);
    return e != cudaSuccess ? e : launch_attn_join(A, bf16, st);
}

}  // namespace gdnspec
