// tree_attn.cu -- attention of a window of drafted tokens over the paged cache on
// the CUDA cores (fp32, and groups of more than 128 heads), and the join of split
// items for both kernels.
//
// Per query row, one pass over the keys with a running maximum m and sum l in
// powers of two: for a tile's scores s (times scale log2 e),
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v,
// and the row's output is o / l.  A row that has seen nothing yet has m = -inf, l = 0.
//
// A block of four or eight warps holds RPT query rows a warp and walks tiles of 32
// keys, copied asynchronously into one of two buffers while the other is worked on.
// For a warp's rows lane k forms the scores with key k (the key row is read once for
// all of them, the query rows are broadcast; key rows are padded by 16 bytes, so
// eight lanes' pieces fall in different banks), the maximum is a shuffle reduction,
// and the sums run over output columns, VEC consecutive ones per lane.  Only the
// buffers are shared between the warps.  It is bound by shared-memory reads: every
// warp reads the whole tile, 8 wavefronts of a key and four query rows for 16
// multiply-adds a lane.
#include "attn_common.cuh"
#include "launch_setup.cuh"

namespace gdnspec {

constexpr int kAttnTile = 32;     // keys of a tile

size_t tree_attn_smem(int D, int MT, int es) {
    const size_t rows = (size_t)kAttnTile * ((D * es + 16) + D * es);          // a tile's keys and values
    return 2 * rows + sizeof(float) * ((size_t)MT * D + MT * (kAttnTile + 4));  // and queries, probabilities
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

// Sixteen bytes from global to shared memory; zeros where !live.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

// W warps of RPT rows (MT = W RPT); NG groups of 32 VEC output columns.
template <typename IO, int W, int RPT, int VEC, int NG>
__global__ void __launch_bounds__(32 * W, 2) tree_attn_kernel(const __grid_constant__ AttnArgs A) {
    constexpr int kAttnThreads = 32 * W, kEach = kAttnThreads / kAttnTile;   // threads that copy a token
    constexpr int MT = W * RPT, PLD = kAttnTile + 4, kPiece = 16 / sizeof(IO);   // elements of 16 bytes
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scratch[kAttnScratch];
    const int D = A.C.D, KLD = D + kPiece;
    IO *const Ks = reinterpret_cast<IO *>(smem);                              // [2][32][D + 16 bytes]
    IO *const Vs = Ks + 2 * kAttnTile * KLD;                                  // [2][32][D]
    float *const Qs = reinterpret_cast<float *>(Vs + 2 * kAttnTile * D);      // [MT][D], times scale log2 e
    float *const Ps = Qs + MT * D;                                            // [MT][36]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x / A.NQT, qt = blockIdx.x - group * A.NQT;
    float *const my_p = Ps + warp * RPT * PLD;
    const float *const my_q = Qs + warp * RPT * D;
    grid_dep_wait();

    attn_dead_rows<IO>(A, blockIdx.x, gridDim.x, tid, kAttnThreads);
    const AttnPlan plan = attn_plan<kAttnThreads>(A, group, blockIdx.x == 0, scratch);
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    bool any = walk.next(A, &pc);
    if (tid == 0 && qt == 0) attn_note(A, group, any, pc, plan.chunk);
    for (; any; any = walk.next(A, &pc)) {
        const int live = min(MT, pc.cnt * A.G - qt * MT);   // rows of this query tile
        if (live <= 0) continue;
        const int kv = pc.len + pc.cnt, pieces = D / kPiece;
        const auto fetch = [&](int t, int buf) {
            const int r = tid / kEach, tok = t * kAttnTile + r;
            int64_t row = -1;
            if (tok < kv) {
                row = kv_token_row(A.C, pc.slot, tok);
                if (row < 0) atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
            }
            const bool there = row >= 0;   // rows past the end are zeros, whatever the page holds there
            const int64_t e = there ? kv_elem(A.C, A.layer, pc.h, row) : 0;
            const IO *k = static_cast<const IO *>(A.C.k) + e, *v = static_cast<const IO *>(A.C.v) + e;
            IO *kd = Ks + (buf * kAttnTile + r) * KLD, *vd = Vs + (buf * kAttnTile + r) * D;
            for (int c = tid % kEach; c < pieces; c += kEach) {
                copy16(kd + c * kPiece, k + c * kPiece, there);
                copy16(vd + c * kPiece, v + c * kPiece, there);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();   // the piece before is done with shared memory
        fetch(pc.t0, 0);
        for (int i = tid; i < MT * D / 4; i += kAttnThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < live) {
                x = load4<IO>(static_cast<const IO *>(A.q) + attn_out_row(A, pc.b, pc.h, qt * MT + r) * D + c);
                x.x *= A.scale_log2, x.y *= A.scale_log2, x.z *= A.scale_log2, x.w *= A.scale_log2;
            }
            *reinterpret_cast<float4 *>(Qs + r * D + c) = x;
        }
        uint64_t mask[RPT];
        float m[RPT], l[RPT];   // l: this lane's keys only, until the end
        float acc[RPT][NG * VEC] = {};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = warp * RPT + i;
            mask[i] = r < live ? attn_mask(A, pc.b, (qt * MT + r) / A.G) : 0;
            m[i] = -INFINITY;
            l[i] = 0.0f;
        }
        for (int t = pc.t0; t < pc.t1; ++t) {
            const int buf = (t - pc.t0) & 1, k0 = t * kAttnTile;
            if (t + 1 < pc.t1) {
                fetch(t + 1, buf ^ 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            const IO *kp = Ks + (buf * kAttnTile + lane) * KLD, *vp = Vs + buf * kAttnTile * D;
            float s[RPT] = {};
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                const float4 kx = load4<IO>(kp + d);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float4 qx = *reinterpret_cast<const float4 *>(my_q + i * D + d);
                    s[i] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, s[i]))));
                }
            }
            const int node = k0 + lane - pc.len;   // < 0: committed
            const bool drafts = k0 + kAttnTile > pc.len;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float x = s[i];
                if (drafts && !(k0 + lane < kv && (node < 0 || ((mask[i] >> node) & 1)))) x = -INFINITY;
                float top = x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float mn = fmaxf(m[i], top), base = mn == -INFINITY ? 0.0f : mn;
                const float p = exp2f(x - base);
                if (mn > m[i]) {   // the same in all lanes
                    const float al = exp2f(m[i] - base);
                    l[i] *= al;
#pragma unroll
                    for (int j = 0; j < NG * VEC; ++j) acc[i][j] *= al;
                    m[i] = mn;
                }
                l[i] += p;
                my_p[i * PLD + lane] = p;
            }
            __syncwarp();
            // A tile that holds drafted tokens leaves masked ones out by a test, so that an infinity or NaN there stays
            // without effect; committed tokens are seen by every row.
#pragma unroll 1
            for (int k = 0; k < kAttnTile; k += 4) {
                float4 p[RPT];
#pragma unroll
                for (int i = 0; i < RPT; ++i) p[i] = *reinterpret_cast<const float4 *>(my_p + i * PLD + k);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v[NG * VEC];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const int d = (g * 32 + lane) * VEC;
                        if (VEC == 4) {
                            const float4 x = d < D ? load4<IO>(vp + (k + e) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[g * VEC] = x.x, v[g * VEC + 1] = x.y, v[g * VEC + 2] = x.z, v[g * VEC + 3] = x.w;
                        } else {
                            const float2 x = d < D ? load2<IO>(vp + (k + e) * D + d) : make_float2(0.f, 0.f);
                            v[g * VEC] = x.x, v[g * VEC + 1] = x.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float x = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                        if (!drafts || x != 0.0f) {
#pragma unroll
                            for (int j = 0; j < NG * VEC; ++j) acc[i][j] = fmaf(x, v[j], acc[i][j]);
                        }
                    }
                }
            }
            __syncthreads();   // the buffer may be filled again
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = warp * RPT + i;
            const float sum = warp_sum(l[i]);
            if (r >= live) continue;
            const int64_t row = attn_out_row(A, pc.b, pc.h, qt * MT + r), part = (int64_t)blockIdx.x * 2 + pc.side;
            const float inv = pc.whole() ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
            IO *out = static_cast<IO *>(A.out) + row * D;
            float *po = reinterpret_cast<float *>(A.part_o) + part * MT * D;
#pragma unroll
            for (int j = 0; j < NG * VEC; ++j) {
                const int d = (j / VEC * 32 + lane) * VEC + j % VEC;
                if (d >= D) continue;
                if (pc.whole()) out[d] = from_f32<IO>(acc[i][j] * inv);
                else po[((d >> 2) * MT + r) * 4 + (d & 3)] = acc[i][j];
            }
            if (lane == 0) {
                if (!pc.whole()) A.part_ml[part * MT + r] = make_float2(m[i], sum);
                else if (A.lse) A.lse[row] = attn_lse(m[i], sum);
            }
        }
    }
    grid_dep_launch();
}

// ------------------------------------------------------------------ join

constexpr int kJoinThreads = 256;
constexpr int kJoinLanes = 8;      // threads that share an element's pieces when they are many
constexpr int kJoinMany = 16;      // from so many pieces on

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

// Block (g, query tile, part).  A thread takes the same four dims of one row from
// every piece, all loads of two pieces in flight before they are merged; where an
// item has many pieces (few rows, long contexts) eight threads share an element.
// Everything about the item is in the chunk's note, so a block starts with one load.
template <typename IO>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs A) {
    __shared__ float4 o_s[kJoinLanes][32];
    __shared__ float2 ml_s[kJoinLanes][32];
    grid_dep_wait();
    const int g = blockIdx.x + 1, qt = blockIdx.y, tid = threadIdx.x, lane = tid & 31, pl = tid >> 5;
    const AttnCut cut = A.cuts[g];
    const int64_t s = (int64_t)g * cut.chunk - cut.t;                // the item's first tile in the line
    if (cut.b < 0 || cut.t == 0 || s / cut.chunk != g - 1) return;   // a cut between items, or not the item's first
    const int live = min(A.MT, cut.cnt * A.G - qt * A.MT);
    if (live <= 0) return;
    const int last = (int)((s + cut.tiles - 1) / cut.chunk);
    const int D4 = A.C.D >> 2, work = live * D4;
    const auto part_of = [&](int c) { return ((int64_t)c * A.NQT + qt) * 2 + (s > (int64_t)c * cut.chunk ? 1 : 0); };
    if (last - g + 2 < kJoinMany) {
        for (int x = blockIdx.z * kJoinThreads + tid; x < work; x += gridDim.z * kJoinThreads) {
            const int d4 = x / live, r = x - d4 * live;
            JoinSum sum;
            for (int c = g - 1; c <= last; c += 2) {
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
    for (int x0 = blockIdx.z * 32; x0 < work; x0 += gridDim.z * 32) {
        const int x = x0 + lane, d4 = x / live, r = x - d4 * live;
        JoinSum sum;
        if (x < work)
            for (int c = g - 1 + pl; c <= last; c += kJoinLanes) {
                const int64_t part = part_of(c);
                sum.add(A.part_ml[part * A.MT + r], A.part_o[(part * D4 + d4) * A.MT + r]);
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

// Rows of a block's query tile: the fewest of 4, 8, 16 and 32 that hold the window.  Sixteen and 32 rows take eight
// warps, which read the tile from shared memory twice as often as four would and cover that latency better: 8
// sequences of 5000 tokens, 4 shared heads of 128 fp32, 8 drafts are 71 us with 16 rows and 108 with 32, against 84
// and 131 with four warps.  Eight rows keep four: 16 of those sequences are 91 us, 100 with eight.
static int tile_rows(int R) { return R <= 4 ? 4 : R <= 8 ? 8 : R <= 16 ? 16 : 32; }

template <typename IO, int W, int RPT, int VEC, int NG>
static cudaError_t run_tree_attn(const AttnArgs &A, cudaStream_t st) {
    static KernelSetup setup;
    const size_t smem = tree_attn_smem(A.C.D, W * RPT, sizeof(IO));
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)tree_attn_kernel<IO, W, RPT, VEC, NG>, smem, &sms);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_attn_kernel<IO, W, RPT, VEC, NG>, dim3(A.groups * A.NQT), dim3(32 * W), smem, st, A);
}

template <typename IO, int W, int RPT>
static cudaError_t run_cols(const AttnArgs &A, cudaStream_t st) {
    if (A.C.D <= 64) return run_tree_attn<IO, W, RPT, 2, 1>(A, st);
    if (A.C.D <= 128) return run_tree_attn<IO, W, RPT, 4, 1>(A, st);
    return run_tree_attn<IO, W, RPT, 4, 2>(A, st);
}

template <typename IO>
static cudaError_t run_rows(const AttnArgs &A, cudaStream_t st) {
    switch (A.MT) {
        case 4: return run_cols<IO, 4, 1>(A, st);
        case 8: return run_cols<IO, 4, 2>(A, st);
        case 16: return run_cols<IO, 8, 2>(A, st);
        default: return run_cols<IO, 8, 4>(A, st);
    }
}

// The cut of the work on a machine of `sms` SMs (MT, TN, NQT, groups).
void tree_attn_cut(AttnArgs *A, int sms, int es) {
    const int R = A->T * A->G;
    A->TN = kAttnTile;
    A->MT = tile_rows(R);
    A->NQT = (R + A->MT - 1) / A->MT;
    int per_sm = (int)((size_t)(227 * 1024) / (tree_attn_smem(A->C.D, A->MT, es) + 2048));
    const int most = A->MT <= 8 ? 4 : 2;
    if (per_sm > most) per_sm = most;
    if (per_sm < 1) per_sm = 1;
    const int groups = sms * per_sm / A->NQT;
    A->groups = groups < 1 ? 1 : groups;
    A->min_chunk = 2;
}

cudaError_t launch_tree_attn(const AttnArgs &A, bool bf16, cudaStream_t st) {
    const cudaError_t e = bf16 ? run_rows<__nv_bfloat16>(A, st) : run_rows<float>(A, st);
    return e != cudaSuccess ? e : launch_attn_join(A, bf16, st);
}

}  // namespace gdnspec
