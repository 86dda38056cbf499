// prompt_attn.cu -- attention of packed prompts over the paged cache on the CUDA cores
// (fp32), and the join of split items for both kernels.
//
// Per query row, one pass over the keys with a running maximum m and sum l in powers of
// two: for a tile's scores s (times scale log2 e),
//   m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),  o' = o 2^(m-m') + sum 2^(s-m') v,
// and the row's output is o / l.  A row that has seen nothing yet has m = -inf, l = 0.
//
// A block holds 64 query rows and walks tiles of 64 keys.  A thread forms the scores of eight rows
// (four where D > 128) with four keys, then, with the probabilities in shared memory where the keys
// were, the sums of the same rows over DP / 16 columns; sixteen threads share the rows.  The
// values are copied while the scores are formed, two blocks an SM cover the rest.  2 prompts of
// 1000 tokens behind 753 and 1000, 8 heads on 2 of 128: 321 us, 35 TFLOP/s, nearly half of the fp32 rate
// (with four rows a thread a tenth slower); heads of 256, 600 tokens: 347 us, 33 TFLOP/s.  What bounds it is latency: two
// warps a scheduler (248 to 255 registers), four block barriers a tile, one buffer each of keys and values.  7 prompts of
// up to 523 tokens behind up to 777, 6 heads on 2 of 64 (91 us): instructions issue in 61% of the active cycles, the
// multiply-adds' pipe is 47% and shared memory's 45% busy; a warp waits for shared memory first, then for what it has
// issued itself, then for instructions and barriers.  Sums are of 64 terms, and of such sums: with one chain a row of 8267
// keys was off by 1.1e-6 of itself, by 3.7e-7 so.
#include "launch_setup.cuh"
#include "prompt_common.cuh"

namespace gdnspec {

constexpr int kPromptRows = 64, kPromptLogTile = 6, kPromptTile = 1 << kPromptLogTile;

// Q and K rows and V rows of a block, in floats; the probabilities lie where the keys were.
constexpr int prompt_q_ld(int DP) { return DP + 4; }
constexpr size_t prompt_smem(int DP) { return sizeof(float) * (size_t)(kPromptRows * prompt_q_ld(DP) + kPromptTile * (prompt_q_ld(DP) + DP)); }

__device__ __forceinline__ void prompt_copy16(void *dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}

// Rows of a thread, threads of a block, and blocks of an SM, as many as the shared memory leaves room for.
constexpr int prompt_rows(int DP) { return DP > 128 ? 4 : 8; }
constexpr int prompt_threads(int DP) { return kPromptRows / prompt_rows(DP) * 16; }
constexpr int prompt_blocks(int DP) { return DP > 128 ? 1 : 2; }

template <int DP>
__global__ void __launch_bounds__(prompt_threads(DP), prompt_blocks(DP)) prompt_attn_kernel(const __grid_constant__ PromptArgs A) {
    constexpr int RT = prompt_rows(DP), kPromptThreads = prompt_threads(DP);
    constexpr int LD = DP + 4, PLD = kPromptTile + 4, NG = DP / 64;   // groups of 64 columns, four of each a thread's
    extern __shared__ __align__(16) float sm[];
    __shared__ PromptScratch scratch;
    __shared__ int64_t elem_s[2][kPromptTile];   // where a tile's keys and values lie in the pool, this one's and the next's
    float *const Qs = sm, *const Ks = Qs + kPromptRows * LD, *const Vs = Ks + kPromptTile * LD, *const Ps = Ks;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, r0 = ty * RT, D = A.C.D, D4 = D >> 2;
    const float *const qg = static_cast<const float *>(A.q);
    grid_dep_wait();

    const PromptPlan plan = prompt_plan<kPromptThreads>(A, &scratch);
    prompt_dead_tokens<float>(A, plan.ascends(), tid, kPromptThreads);
    PromptWalk walk(A, plan, 0);   // (one wave: the keys and values are not what bounds it)
    if (tid == 0) prompt_note(A, walk, plan.chunk, 0);
    PromptPiece pc;
    while (walk.next(A, plan, &pc)) {
        const PromptItem &it = pc.it;
        __syncthreads();   // the piece before is done with shared memory
        for (int x = tid; x < kPromptRows * (DP / 4); x += kPromptThreads) {
            const int r = x / (DP / 4), d = x % (DP / 4) * 4;
            bool on;
            const int64_t row = prompt_out_row(A, it, r, &on);
            on = on && d < D;
            prompt_copy16(Qs + r * LD + d, qg + (on ? row * D + d : 0), on);
        }
        int see[RT];   // keys that the thread's rows attend to
        float m[RT], l[RT], acc[RT][NG * 4] = {};
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            bool on;
            prompt_out_row(A, it, r0 + i, &on);
            see[i] = on ? it.len + it.q0 + (r0 + i) / A.GS + 1 : 0;
            m[i] = -INFINITY;
            l[i] = 0.0f;
        }
        const int all = it.len + it.q0 + 1;   // keys that every row attends to
        const auto look_up = [&](int t) {
            if (tid < kPromptTile && t < pc.t1) {
                int64_t e = -1;
                if (t * kPromptTile + tid < it.keys) {
                    const int64_t row = kv_token_row(A.C, it.slot, t * kPromptTile + tid);
                    if (row < 0) atomicOr(A.C.status, GDN_SPEC_ST_PAGE_OOR);
                    else e = kv_elem(A.C, A.layer, it.h, row);
                }
                elem_s[t & 1][tid] = e;
            }
        };
        look_up(pc.t0);
        for (int t = pc.t0; t < pc.t1; ++t) {
            const int k0 = t * kPromptTile;
            const bool edge = k0 + kPromptTile > all;
            __syncthreads();   // the tile before is done with
            // rows past the end are zeros; the values are on their way while the scores are formed
            const auto fetch = [&](float *to, int ld, const void *pool) {
#pragma unroll 4
                for (int x = tid; x < kPromptTile * (DP / 4); x += kPromptThreads) {
                    const int r = x / (DP / 4), d = x % (DP / 4) * 4;
                    const int64_t e = elem_s[t & 1][r];
                    const bool on = e >= 0 && d < D;
                    prompt_copy16(to + r * ld + d, static_cast<const float *>(pool) + (on ? e + d : 0), on);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            fetch(Ks, LD, A.C.k);
            fetch(Vs, DP, A.C.v);
            look_up(t + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            float s[RT][4] = {};
#pragma unroll 1
            for (int d0 = 0; d0 < DP; d0 += 64) {
                float u[RT][4] = {};
#pragma unroll 4
                for (int d = d0; d < d0 + 64; d += 4) {
                    float4 k[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * j) * LD + d);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float4 q = *reinterpret_cast<const float4 *>(Qs + (r0 + i) * LD + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            u[i][j] = fmaf(q.x, k[j].x, u[i][j]);
                            u[i][j] = fmaf(q.y, k[j].y, u[i][j]);
                            u[i][j] = fmaf(q.z, k[j].z, u[i][j]);
                            u[i][j] = fmaf(q.w, k[j].w, u[i][j]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] += u[i][j];
            }
            __syncthreads();   // the keys are done with: the probabilities take their place
            float al[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = edge && k0 + tx + 16 * j >= see[i] ? -INFINITY : s[i][j] * A.scale_log2;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float mn = fmaxf(m[i], top), base = mn == -INFINITY ? 0.0f : mn;
                al[i] = exp2f(m[i] - base);
                m[i] = mn;
                l[i] *= al[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(s[i][j] - base);
                    l[i] += p;   // this thread's keys only, until the end
                    Ps[(r0 + i) * PLD + tx + 16 * j] = p;
                }
            }
            // a row's probabilities are read by the half warp that wrote them, the values by all
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            // In a tile that some row does not see all of, masked keys are left out by a test, so that an infinity or
            // NaN there stays without effect.  (By their place: a weight of zero may be one that vanished, and an
            // infinite value is not lost beside it.  Heads of 128: 315 -> 321 us; with a mark below zero in the weight's
            // place 329.)
            float sum[RT][NG * 4] = {};   // over the tile
            const auto add = [&](auto test) {
#pragma unroll 2
                for (int k = 0; k < kPromptTile; k += 4) {
                    float4 p[RT];
#pragma unroll
                    for (int i = 0; i < RT; ++i) p[i] = *reinterpret_cast<const float4 *>(Ps + (r0 + i) * PLD + k);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const float4 v = *reinterpret_cast<const float4 *>(Vs + (k + e) * DP + g * 64 + tx * 4);
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                const float x = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                                if (decltype(test)::value && k0 + k + e >= see[i]) continue;
                                sum[i][g * 4] = fmaf(x, v.x, sum[i][g * 4]);
                                sum[i][g * 4 + 1] = fmaf(x, v.y, sum[i][g * 4 + 1]);
                                sum[i][g * 4 + 2] = fmaf(x, v.z, sum[i][g * 4 + 2]);
                                sum[i][g * 4 + 3] = fmaf(x, v.w, sum[i][g * 4 + 3]);
                            }
                        }
                }
            };
            if (edge) add(std::true_type());
            else add(std::false_type());
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < NG * 4; ++j) acc[i][j] = fmaf(acc[i][j], al[i], sum[i][j]);
        }
        const int64_t part = (int64_t)blockIdx.x * 2 + pc.side();
#pragma unroll
        for (int i = 0; i < RT; ++i) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            bool on;
            const int64_t row = prompt_out_row(A, it, r0 + i, &on);
            if (!on) continue;
            const float inv = 1.0f / l[i];   // (no weight at all, every score -inf: infinite, and zeros times it are NaN)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int d = g * 64 + tx * 4;
                if (d >= D) continue;
                const float *a = acc[i] + g * 4;
                if (pc.whole())
                    *reinterpret_cast<float4 *>(static_cast<float *>(A.out) + row * D + d) =
                        make_float4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
                else
                    A.part_o[(part * D4 + d / 4) * A.MT + r0 + i] = make_float4(a[0], a[1], a[2], a[3]);
            }
            if (tx == 0) {
                if (!pc.whole()) A.part_ml[part * A.MT + r0 + i] = make_float2(m[i], l[i]);
                else if (A.lse) A.lse[row] = attn_lse(m[i], l[i]);
            }
        }
    }
    grid_dep_launch();
}

// ------------------------------------------------------------------ join

constexpr int kPromptJoinThreads = 256;

// Block (g, part), for the item that chunk g starts inside of; the blocks of all chunks that do share the item's
// elements.  A thread takes the same four dims of one row from every piece, in order.
template <typename IO>
__global__ void __launch_bounds__(kPromptJoinThreads) prompt_join_kernel(const __grid_constant__ PromptArgs A) {
    grid_dep_wait();
    const int g = blockIdx.x + 1;
    const PromptCut cut = A.cuts[g];
    const PromptItem &it = cut.item;
    if (it.b < 0) return;
    if (it.tile_at(A, (int64_t)g * cut.chunk) == 0) return;   // a cut between items
    // the cuts inside the item: from the first that leaves a tile before it on
    const int64_t begin = it.pos + A.gap;
    const int first = (int)((begin + (1 << A.log_tn) + cut.chunk - 1) / cut.chunk) - 1, last = (int)((begin + it.keys - 1) / cut.chunk);
    const int D4 = A.C.D >> 2, rows = min(A.tokens, it.cnt - it.q0) * A.GS, work = rows * D4;
    const int block = (g - 1 - first) * gridDim.y + blockIdx.y, blocks = (last - first) * gridDim.y;   // of the item
    for (int x = block * kPromptJoinThreads + threadIdx.x; x < work; x += blocks * kPromptJoinThreads) {
        const int d4 = x / rows, r = x - d4 * rows;
        bool on;
        const int64_t row = prompt_out_row(A, it, r, &on);
        if (!on) continue;
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = first; c <= last; ++c) {
            const int64_t part = (int64_t)c * 2 + (c == first ? 1 : 0);
            const float2 ml = A.part_ml[part * A.MT + r];
            const float4 po = A.part_o[(part * D4 + d4) * A.MT + r];
            if (ml.y == 0.0f) continue;   // that piece saw nothing, its sums may be anything
            const float mn = fmaxf(m, ml.x), wa = exp2f(m - mn), wb = exp2f(ml.x - mn);
            l = l * wa + ml.y * wb;
            o.x = o.x * wa + po.x * wb;
            o.y = o.y * wa + po.y * wb;
            o.z = o.z * wa + po.z * wb;
            o.w = o.w * wa + po.w * wb;
            m = mn;
        }
        const float inv = 1.0f / l;   // (as in the kernels: NaN where every score is -inf)
        IO out[4] = {from_f32<IO>(o.x * inv), from_f32<IO>(o.y * inv), from_f32<IO>(o.z * inv), from_f32<IO>(o.w * inv)};
        IO *op = static_cast<IO *>(A.out) + row * A.C.D + 4 * d4;
        if (sizeof(IO) == 2) *reinterpret_cast<uint2 *>(op) = *reinterpret_cast<const uint2 *>(out);
        else *reinterpret_cast<uint4 *>(op) = *reinterpret_cast<const uint4 *>(out);
        if (A.lse && d4 == 0) A.lse[row] = attn_lse(m, l);
    }
}

cudaError_t launch_prompt_join(const PromptArgs &A, bool bf16, cudaStream_t stream) {
    const int chunks = A.groups * A.waves;
    if (chunks < 2) return cudaSuccess;
    const dim3 grid(chunks - 1, A.waves > 1 ? 4 : 8);   // (most cuts of many are one of a few pieces' item)
    return bf16 ? launch_dependent(prompt_join_kernel<__nv_bfloat16>, grid, dim3(kPromptJoinThreads), 0, stream, A)
                : launch_dependent(prompt_join_kernel<float>, grid, dim3(kPromptJoinThreads), 0, stream, A);
}

// ------------------------------------------------------------------ launch

template <int DP>
static cudaError_t run_prompt_attn(const PromptArgs &A, cudaStream_t st) {
    static KernelSetup setup;
    int sms;
    const cudaError_t e = kernel_setup(setup, (const void *)prompt_attn_kernel<DP>, prompt_smem(DP), &sms);
    if (e != cudaSuccess) return e;
    return launch_dependent(prompt_attn_kernel<DP>, dim3(A.groups), dim3(prompt_threads(DP)), prompt_smem(DP), st, A);
}

// The cut of the work on a machine of `sms` SMs.
void prompt_attn_cut(PromptArgs *A, int sms) {
    A->log_tn = kPromptLogTile;
    A->MT = kPromptRows;
    A->HS = (A->G + A->MT - 1) / A->MT;
    A->GS = (A->G + A->HS - 1) / A->HS;
    A->tokens = A->MT / A->GS;
    A->groups = sms * prompt_blocks(A->C.D);
    A->waves = 1;
    A->gap = kPromptTile;
}

cudaError_t launch_prompt_attn(const PromptArgs &A, cudaStream_t st) {
    const cudaError_t e = A.C.D <= 64 ? run_prompt_attn<64>(A, st) : A.C.D <= 128 ? run_prompt_attn<128>(A, st) : run_prompt_attn<256>(A, st);
    return e != cudaSuccess ? e : launch_prompt_join(A, false, st);
}

}  // namespace gdnspec
