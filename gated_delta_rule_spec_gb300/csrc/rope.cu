// rope.cu -- rotary positions: of a tensor (and their transpose, the gradient),
// and of a window's q and k together with the append of k and v to the paged
// cache.
//
// Pair i of a head is turned by the angle pos * f_i.  The plan holds f_i as a
// fraction of 2^64 of a turn, so pos * freq modulo 2^64 is the angle modulo a
// turn, exact to 2^-64 pos: the reduction costs one integer product and loses
// nothing at long positions, where the fp32 product pos * f_i would be off by
// 2^-24 of the whole angle.  sincospi of the signed fraction gives cos and sin to
// fp32 accuracy.  No table of positions is kept.
//
// Bound by HBM: every q, k, v element is read once and written once.  A block takes
// one to sixteen tokens: its threads first form the tokens' cos and sin
// (rot / 2 pairs a token, shared by all heads) in shared memory, then turn 16
// elements of one head each (two runs of 8, a pair's halves in the half
// layout).  The SM's other blocks cover a block's set-up, so registers are held to
// eight blocks an SM in bf16 (128 windows of 8 tokens, 16 + 2 x 2 heads of 256: 5.8 us,
// 7.3 with five) and six in fp32; loading a thread's next unit before this one's
// arithmetic took the registers for that and was slower (some of the kernels keep 4 to 24
// bytes a thread in local memory at that).  8 x 4096 tokens, 32 + 2 x 8
// heads of 128, bf16: 124 us, 0.96 of the copy bandwidth (134 us with a token's cos
// and sin in the order of the pairs, where a warp's reads met in the same banks).
#include "kv_common.cuh"
#include "launch_setup.cuh"
#include "rope_common.cuh"

namespace gdnspec {

__host__ __device__ constexpr int rope_blocks(size_t es) { return es == 2 ? 8 : 6; }   // of an SM

// x and out may be the same memory (each unit reads what it writes, before it
// writes), so neither is __restrict__.
template <typename IO, bool HALF, bool UNITS>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks(sizeof(IO))) rope_kernel(const __grid_constant__ RopeArgs R, int N, int heads, int tokens,
                                                            const int32_t *__restrict__ pos, const IO *x,
                                                            int64_t x_stride, IO *out, int64_t out_stride, float sign) {
    extern __shared__ __align__(16) float2 cs[];   // [tokens][pairs], see turn_place
    const int n0 = blockIdx.x * tokens, tid = threadIdx.x;
    const int live = min(tokens, N - n0);
    grid_dep_wait();
    for (int j = tid; j < live * R.pairs; j += kRopeThreads) {
        const int t = j / R.pairs, i = j - t * R.pairs;
        cs[t * R.pairs + turn_place<UNITS>(i, R.pairs)] = rope_turn(R, pos[n0 + t], i);
    }
    __syncthreads();
    if (UNITS) {
        const int per_head = R.D >> 4, per_token = heads * per_head, turning = R.rot >> 4;
        for (int j = tid; j < live * per_token; j += kRopeThreads) {
            const int t = j / per_token, r = j - t * per_token, h = r / per_head, u = r - h * per_head;
            int o0, o1;
            unit_runs<HALF>(u, R.rot, &o0, &o1);
            const IO *xp = x + (n0 + t) * x_stride + h * R.D;
            IO *op = out + (n0 + t) * out_stride + h * R.D;
            Run8<IO> r0, r1;
            r0.load(xp + o0);
            r1.load(xp + o1);
            if (u < turning) turn_unit<IO, HALF>(r0, r1, cs + t * R.pairs, u, R.pairs, sign);
            r0.store(op + o0);
            r1.store(op + o1);
        }
    } else {
        const int per_head = R.D - R.pairs, per_token = heads * per_head;
        for (int j = tid; j < live * per_token; j += kRopeThreads) {
            const int t = j / per_token, r = j - t * per_token, h = r / per_head, e = r - h * per_head;
            turn_scalar<IO, HALF>(x + (n0 + t) * x_stride + h * R.D, out + (n0 + t) * out_stride + h * R.D, cs + t * R.pairs,
                                  R.rot, R.D, sign, e);
        }
    }
}

// A window's tokens: q turned into q_out, k turned and v copied into the pages.
// Token j of the launch is (row j / T, t = j % T).  What becomes of it (where its
// key goes, or that it is dead) is decided by one thread per token beside the
// cos and sin.  A table entry that is no page is the matter of the tokens that would
// lie in it: refusing their whole row would have every block look at all the row's
// entries (92 x 2524 tokens of 10 heads of 64 in pages of 16: 121 us as it is, 138 so;
// 128 windows of 8: 6.4 and 7.2 us).
template <typename IO, bool HALF, bool UNITS>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks(sizeof(IO))) rope_append_kernel(
    const __grid_constant__ RopeArgs R, const __grid_constant__ KvArgs C, int layer, int B, int T, int tokens, int HQ,
    const int32_t *__restrict__ slot_idx, const int32_t *__restrict__ n_tokens, const int32_t *__restrict__ pos,
    const IO *__restrict__ q, int64_t q_stride, const IO *__restrict__ k, int64_t k_stride, const IO *__restrict__ v,
    int64_t v_stride, IO *__restrict__ q_out) {
    extern __shared__ __align__(16) float2 cs[];   // [tokens][pairs], see turn_place
    __shared__ int64_t row_s[kRopeTokens];   // the token's row in the pool, -1: its q is zero and nothing is written
    __shared__ int pos_s[kRopeTokens];
    const int tid = threadIdx.x;
    const int64_t all = (int64_t)B * T, j0 = (int64_t)blockIdx.x * tokens;
    const int live = (int)min((int64_t)tokens, all - j0);
    grid_dep_wait();
    if (tid < live) {
        const int b = (int)((j0 + tid) / T), t = (int)(j0 + tid - (int64_t)b * T);
        const int slot = slot_idx[b], cnt = n_tokens ? n_tokens[b] : T;
        uint32_t bits;
        const int len = kv_row(C, slot, cnt, T, &bits);
        int64_t row = -1;
        if (len >= 0 && t < cnt) {
            row = kv_token_row(C, slot, len + t);
            if (row < 0) bits |= GDN_SPEC_ST_PAGE_OOR;
        }
        if (bits) atomicOr(C.status, bits);
        row_s[tid] = row;
        pos_s[tid] = pos ? pos[j0 + tid] : len + t;
    }
    __syncthreads();
    for (int j = tid; j < live * R.pairs; j += kRopeThreads) {
        const int t = j / R.pairs, i = j - t * R.pairs;
        cs[t * R.pairs + turn_place<UNITS>(i, R.pairs)] = rope_turn(R, pos_s[t], i);
    }
    __syncthreads();
    const int heads = HQ + 2 * C.HKV;
    const int per_head = UNITS ? R.D >> 4 : R.D - R.pairs, per_token = heads * per_head, turning = R.rot >> 4;
    IO *kp = static_cast<IO *>(C.k), *vp = static_cast<IO *>(C.v);
    for (int j = tid; j < live * per_token; j += kRopeThreads) {
        const int t = j / per_token, r = j - t * per_token, h = r / per_head, u = r - h * per_head;
        const int64_t token = j0 + t, row = row_s[t];
        const IO *src;
        IO *dst;
        if (h < HQ) {
            src = q + token * q_stride + h * R.D;
            dst = q_out + (token * HQ + h) * R.D;
        } else if (row < 0) {
            continue;
        } else if (h < HQ + C.HKV) {
            src = k + token * k_stride + (h - HQ) * R.D;
            dst = kp + kv_elem(C, layer, h - HQ, row);
        } else {
            src = v + token * v_stride + (h - HQ - C.HKV) * R.D;
            dst = vp + kv_elem(C, layer, h - HQ - C.HKV, row);
        }
        const bool is_v = h >= HQ + C.HKV;
        if (UNITS) {
            int o0, o1;
            unit_runs<HALF>(u, R.rot, &o0, &o1);
            Run8<IO> r0, r1;
            if (row < 0) {
                r0.zero();
                r1.zero();
            } else {
                r0.load(src + o0);
                r1.load(src + o1);
                if (u < turning && !is_v) turn_unit<IO, HALF>(r0, r1, cs + t * R.pairs, u, R.pairs, 1.0f);
            }
            r0.store(dst + o0);
            r1.store(dst + o1);
        } else if (row < 0 || is_v) {
            // the elements that turn_scalar would write for u
            const int i0 = u < R.pairs ? (HALF ? u : 2 * u) : R.rot + u - R.pairs;
            dst[i0] = row < 0 ? from_f32<IO>(0.0f) : src[i0];
            if (u < R.pairs) {
                const int i1 = HALF ? u + R.pairs : 2 * u + 1;
                dst[i1] = row < 0 ? from_f32<IO>(0.0f) : src[i1];
            }
        } else {
            turn_scalar<IO, HALF>(src, dst, cs + t * R.pairs, R.rot, R.D, 1.0f, u);
        }
    }
}

// Four tokens a block once that still gives every SM several blocks, and more while they do not fill the block's threads
// twice (n tokens of `units` units each).  82 x 725 tokens, 6 + 2 x 2 heads of 128 bf16, 80 units: 71 us with four, 63
// with eight; 54 x 1141 tokens, 3 + 2 heads of 64, 20 units: 37 us with four, 27 with sixteen.
static int tokens_per_block(int64_t n, int units) {
    int t = n >= 4096 ? 4 : 1;
    while (t >= 4 && t < kRopeTokens && t * units < 2 * kRopeThreads && n >= 4096 * t) t *= 2;
    return t;
}

template <typename IO, bool HALF, bool UNITS>
static cudaError_t run_rope(const RopeArgs &R, int N, int heads, const int32_t *pos, const void *x, int64_t x_stride,
                            void *out, int64_t out_stride, bool transpose, cudaStream_t st) {
    const int tokens = tokens_per_block(N, heads * R.D / 16);
    const int64_t blocks = ((int64_t)N + tokens - 1) / tokens;
    return launch_dependent(rope_kernel<IO, HALF, UNITS>, dim3((unsigned)blocks), dim3(kRopeThreads),
                            tokens * R.pairs * sizeof(float2), st, R, N, heads, tokens, pos, static_cast<const IO *>(x), x_stride,
                            static_cast<IO *>(out), out_stride, transpose ? -1.0f : 1.0f);
}

cudaError_t launch_rope(const gdn_spec_rope_plan *plan, int N, int heads, bool bf16, const int32_t *pos, const void *x,
                        int64_t x_stride, void *out, int64_t out_stride, bool transpose, cudaStream_t st) {
    const RopeArgs R = rope_args(plan);
    const bool half = plan->layout == GDN_SPEC_ROPE_HALF, units = plan->D % 16 == 0 && plan->rot % 16 == 0;
    const auto go = [&](auto kern) { return kern(R, N, heads, pos, x, x_stride, out, out_stride, transpose, st); };
    if (bf16) {
        if (units) return half ? go(run_rope<__nv_bfloat16, true, true>) : go(run_rope<__nv_bfloat16, false, true>);
        return half ? go(run_rope<__nv_bfloat16, true, false>) : go(run_rope<__nv_bfloat16, false, false>);
    }
    if (units) return half ? go(run_rope<float, true, true>) : go(run_rope<float, false, true>);
    return half ? go(run_rope<float, true, false>) : go(run_rope<float, false, false>);
}

template <typename IO, bool HALF, bool UNITS>
static cudaError_t run_append(const RopeArgs &R, const KvArgs &C, int layer, const int32_t *slot_idx, int B, int T,
                              const int32_t *n_tokens, const int32_t *pos, int HQ, const void *q, int64_t q_stride,
                              const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *q_out,
                              cudaStream_t st) {
    const int64_t all = (int64_t)B * T;
    const int tokens = tokens_per_block(all, (HQ + 2 * C.HKV) * C.D / 16);
    return launch_dependent(rope_append_kernel<IO, HALF, UNITS>, dim3((unsigned)((all + tokens - 1) / tokens)),
                            dim3(kRopeThreads), tokens * R.pairs * sizeof(float2), st, R, C, layer, B, T, tokens, HQ, slot_idx, n_tokens, pos,
                            static_cast<const IO *>(q), q_stride, static_cast<const IO *>(k), k_stride,
                            static_cast<const IO *>(v), v_stride, static_cast<IO *>(q_out));
}

cudaError_t launch_rope_append(const gdn_spec_rope_plan *plan, const KvArgs &C, bool bf16, int layer,
                               const int32_t *slot_idx, int B, int T, const int32_t *n_tokens, const int32_t *pos, int HQ,
                               const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, void *q_out, cudaStream_t st) {
    const RopeArgs R = rope_args(plan);
    const bool half = plan->layout == GDN_SPEC_ROPE_HALF, units = plan->D % 16 == 0 && plan->rot % 16 == 0;
    const auto go = [&](auto kern) {
        return kern(R, C, layer, slot_idx, B, T, n_tokens, pos, HQ, q, q_stride, k, k_stride, v, v_stride, q_out, st);
    };
    if (bf16) {
        if (units) return half ? go(run_append<__nv_bfloat16, true, true>) : go(run_append<__nv_bfloat16, false, true>);
        return half ? go(run_append<__nv_bfloat16, true, false>) : go(run_append<__nv_bfloat16, false, false>);
    }
    if (units) return half ? go(run_append<float, true, true>) : go(run_append<float, false, true>);
    return half ? go(run_append<float, true, false>) : go(run_append<float, false, false>);
}

}  // namespace gdnspec
