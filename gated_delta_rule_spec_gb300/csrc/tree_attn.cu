// tree_attn.cu -- attention of a window of drafted tokens over the paged cache on
// the CUDA cores (fp32, and head dims that the tensor-core kernel does not take),
// and the join of split items for both kernels.
//
// Per query row, one pass over the keys with a running maximum m and sum l in
// powers of two: for a tile's scores s (times scale log2 e),
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v,
// and the row's output is o / l.  A row that has seen nothing yet has m = -inf, l = 0.
//
// A block of 256 threads holds MT = 4 RPT query rows and walks tiles of 64 keys
// held in shared memory in fp32.  Scores: thread (i, c) forms those of key c with
// its RPT rows, the key read once and the query rows broadcast, so a key's 16 bytes
// serve RPT rows; the key rows are padded by 16 bytes so that eight keys' pieces
// fall in different banks.  Sums: the same thread layout over output columns.
// Shared-memory reads bound it (12 wavefronts for the 8 cycles of FMA that 32
// multiply-adds take at RPT = 8); with few rows it is bound by the loads.
#include "attn_common.cuh"
#include "launch_setup.cuh"

namespace gdnspec {

constexpr int kAttnThreads = 256;
constexpr int kAttnTile = 64;     // keys of a tile

__host__ __device__ constexpr int attn_key_ld(int D) { return D + 4; }

size_t tree_attn_smem(int D, int MT) {
    return sizeof(float) * ((size_t)MT * D + kAttnTile * attn_key_ld(D) + kAttnTile * D + MT * (kAttnTile + 4) + 3 * MT);
}

template <typename IO> __device__ __forceinline__ void load8(const IO *p, float (&x)[8]);
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// RPT rows per thread (MT = 4 RPT), COLS = ceil(D / 64) output columns per thread.
template <typename IO, int RPT, int COLS>
__global__ void __launch_bounds__(kAttnThreads) tree_attn_kernel(const __grid_constant__ AttnArgs A) {
    constexpr int MT = 4 * RPT, SLD = kAttnTile + 4;
    extern __shared__ float sm[];
    __shared__ int scratch[kAttnScratch];
    const int D = A.C.D, KLD = attn_key_ld(D);
    float *const Qs = sm;                        // [MT][D], times scale log2 e
    float *const Ks = Qs + MT * D;               // [64][D + 4]
    float *const Vs = Ks + kAttnTile * KLD;      // [64][D]
    float *const Ss = Vs + kAttnTile * D;        // [MT][68] scores, then probabilities
    float *const m_s = Ss + MT * SLD, *const l_s = m_s + MT, *const a_s = l_s + MT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = tid >> 6, c64 = tid & 63;     // rows rg * RPT .., key or column c64
    const int group = blockIdx.x / A.NQT, qt = blockIdx.x - group * A.NQT;

    attn_dead_rows<IO>(A, blockIdx.x, gridDim.x, kAttnThreads);
    const AttnPlan plan = attn_plan<kAttnThreads>(A, group, blockIdx.x == 0, scratch);
    AttnWalk walk = attn_walk(A, plan, group);
    AttnPiece pc;
    bool any = walk.next(A, &pc);
    if (tid == 0 && qt == 0) attn_note(A, group, any, pc, plan.chunk);
    for (; any; any = walk.next(A, &pc)) {
        const int live = min(MT, pc.cnt * A.G - qt * MT);   // rows of this query tile
        if (live <= 0) continue;
        const int kv = pc.len + pc.cnt, D8 = D >> 3;
        __syncthreads();   // the piece before is done with shared memory
        for (int i = tid; i < MT * D8; i += kAttnThreads) {
            const int r = i / D8, c = (i - r * D8) * 8;
            float x[8] = {};
            if (r < live) {
                load8<IO>(static_cast<const IO *>(A.q) + attn_out_row(A, pc.b, pc.h, qt * MT + r) * D + c, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= A.scale_log2;
            }
            store8(Qs + r * D + c, x);
        }
        if (tid < MT) {
            m_s[tid] = -INFINITY;
            l_s[tid] = 0.0f;
        }
        float acc[RPT][COLS] = {};
        for (int t = pc.t0; t < pc.t1; ++t) {
            const int k0 = t * kAttnTile, n = min(kAttnTile, kv - k0);
            __syncthreads();
            for (int i = tid; i < kAttnTile * D8; i += kAttnThreads) {
                const int r = i / D8, c = (i - r * D8) * 8;
                float kx[8] = {}, vx[8] = {};
                if (r < n) {   // rows past the end are zeros, whatever the page holds there
                    const int64_t row = kv_token_row(A.C, pc.slot, k0 + r);
                    if (row >= 0) {
                        const int64_t e = kv_elem(A.C, A.layer, pc.h, row) + c;
                        load8<IO>(static_cast<const IO *>(A.C.k) + e, kx);
                        load8<IO>(static_cast<const IO *>(A.C.v) + e, vx);
                    } else if (c == 0) {
                        atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
                    }
                }
                store8(Ks + r * KLD + c, kx);
                store8(Vs + r * D + c, vx);
            }
            __syncthreads();
            {   // scores of key c64
                float s[RPT] = {};
                const float *kp = Ks + c64 * KLD, *qp = Qs + rg * RPT * D;
                for (int d = 0; d < D; d += 4) {
                    const float4 kx = *reinterpret_cast<const float4 *>(kp + d);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float4 qx = *reinterpret_cast<const float4 *>(qp + i * D + d);
                        s[i] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, s[i]))));
                    }
                }
                const int node = k0 + c64 - pc.len;
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int r = rg * RPT + i;
                    bool seen = c64 < n && r < live;
                    if (seen && node >= 0) seen = (attn_mask(A, pc.b, (qt * MT + r) / A.G) >> node) & 1;
                    Ss[r * SLD + c64] = seen ? s[i] : -INFINITY;
                }
            }
            __syncthreads();
            for (int r = warp; r < MT; r += kAttnThreads / 32) {
                float *sp = Ss + r * SLD;
                const float x0 = sp[lane], x1 = sp[lane + 32], m = m_s[r];
                float mx = fmaxf(x0, x1);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.0f : mn;
                const float p0 = exp2f(x0 - base), p1 = exp2f(x1 - base);
                const float sum = warp_sum(p0 + p1), al = exp2f(m - base);
                sp[lane] = p0;
                sp[lane + 32] = p1;
                if (lane == 0) {
                    m_s[r] = mn;
                    l_s[r] = l_s[r] * al + sum;
                    a_s[r] = al;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float al = a_s[rg * RPT + i];
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[i][j] *= al;
            }
            // A tile that holds drafted tokens leaves masked ones out by a test, so that an infinity or
            // NaN there stays without effect; committed tokens are seen by every row.
            const bool drafts = k0 + n > pc.len;
            for (int c = 0; c < kAttnTile; c += 4) {
                float4 p[RPT];
#pragma unroll
                for (int i = 0; i < RPT; ++i) p[i] = *reinterpret_cast<const float4 *>(Ss + (rg * RPT + i) * SLD + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v[COLS];
#pragma unroll
                    for (int j = 0; j < COLS; ++j) {
                        const int d = c64 + 64 * j;
                        v[j] = d < D ? Vs[(c + e) * D + d] : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float x = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                        if (drafts) {
                            if (x != 0.0f)
#pragma unroll
                                for (int j = 0; j < COLS; ++j) acc[i][j] = fmaf(x, v[j], acc[i][j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < COLS; ++j) acc[i][j] = fmaf(x, v[j], acc[i][j]);
                        }
                    }
                }
            }
        }
        // l_s and m_s were written before the barrier in front of the last sums
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg * RPT + i;
            if (r >= live) continue;
            const float l = l_s[r];
            if (pc.whole()) {
                const int64_t row = attn_out_row(A, pc.b, pc.h, qt * MT + r);
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
                for (int j = 0; j < COLS; ++j) {
                    const int d = c64 + 64 * j;
                    if (d < D) static_cast<IO *>(A.out)[row * D + d] = from_f32<IO>(acc[i][j] * inv);
                }
                if (A.lse && c64 == 0) A.lse[row] = attn_lse(m_s[r], l);
            } else {
                const int64_t part = (int64_t)blockIdx.x * 2 + pc.side;
                float *po = reinterpret_cast<float *>(A.part_o) + part * MT * D;
#pragma unroll
                for (int j = 0; j < COLS; ++j) {
                    const int d = c64 + 64 * j;
                    if (d < D) po[((d >> 2) * MT + r) * 4 + (d & 3)] = acc[i][j];
                }
                if (c64 == 0) A.part_ml[part * MT + r] = make_float2(m_s[r], l);
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

// Rows of a block's query tile: the fewest that hold the window, at most 32.
static int rows_per_thread(int R) { return R <= 4 ? 1 : R <= 8 ? 2 : R <= 16 ? 4 : 8; }

template <typename IO, int RPT, int COLS>
static cudaError_t run_tree_attn(const AttnArgs &A, cudaStream_t st) {
    static KernelSetup setup;
    const size_t smem = tree_attn_smem(A.C.D, 4 * RPT);
    int sms;
    cudaError_t e = kernel_setup(setup, (const void *)tree_attn_kernel<IO, RPT, COLS>, smem, &sms);
    if (e != cudaSuccess) return e;
    tree_attn_kernel<IO, RPT, COLS><<<A.groups * A.NQT, kAttnThreads, smem, st>>>(A);
    return cudaGetLastError();
}

template <typename IO, int RPT>
static cudaError_t run_cols(const AttnArgs &A, cudaStream_t st) {
    switch ((A.C.D + 63) / 64) {
        case 1: return run_tree_attn<IO, RPT, 1>(A, st);
        case 2: return run_tree_attn<IO, RPT, 2>(A, st);
        case 3: return run_tree_attn<IO, RPT, 3>(A, st);
        default: return run_tree_attn<IO, RPT, 4>(A, st);
    }
}

template <typename IO>
static cudaError_t run_rows(const AttnArgs &A, cudaStream_t st) {
    switch (A.MT) {
        case 4: return run_cols<IO, 1>(A, st);
        case 8: return run_cols<IO, 2>(A, st);
        case 16: return run_cols<IO, 4>(A, st);
        default: return run_cols<IO, 8>(A, st);
    }
}

// The cut of the work on a machine of `sms` SMs (MT, TN, NQT, groups).
void tree_attn_cut(AttnArgs *A, int sms) {
    const int R = A->T * A->G;
    A->TN = kAttnTile;
    A->MT = 4 * rows_per_thread(R);
    A->NQT = (R + A->MT - 1) / A->MT;
    int per_sm = (int)((size_t)(228 * 1024) / (tree_attn_smem(A->C.D, A->MT) + 1024));
    if (per_sm > 4) per_sm = 4;
    if (per_sm < 1) per_sm = 1;
    const int groups = sms * per_sm / A->NQT;
    A->groups = groups < 1 ? 1 : groups;
    A->min_chunk = 1;
}

cudaError_t launch_tree_attn(const AttnArgs &A, bool bf16, cudaStream_t st) {
    const cudaError_t e = bf16 ? run_rows<__nv_bfloat16>(A, st) : run_rows<float>(A, st);
    return e != cudaSuccess ? e : launch_attn_join(A, bf16, st);
}

}  // namespace gdnspec
