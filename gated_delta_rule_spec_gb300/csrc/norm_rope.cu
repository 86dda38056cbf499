// norm_rope.cu -- the norm of every head with its rotary position in one pass: of a
// tensor, of packed prompts' q and k together with the append of k and v to the paged
// cache, and the gradient.
//
//   y = R(pos) (r x * w),   r = 1 / sqrt(mean(x^2) + eps),   w = weight + offset
// with R the turn of rope_common.cuh.  From dy, with g = R^T dy (the turn back):
//   dx = r (w g - r^2 x mean(w g x)),   dw = sum over tokens and heads of r x g
//
// Bound by HBM: every element is read once and written once.  A block takes some tokens: its
// threads form their cos and sin and the weights in shared memory, then 2^k threads
// take a head, 16 elements each (two runs of 8, a pair's halves in the half layout), so the
// mean is a shuffle over them and a head is never read twice.  Heads of other than 1, 2, 4, 8
// or 16 units leave some of the 2^k idle.  Dims that do not come in units of 16 go element by
// element, a warp a head.  A head's elements are loaded a step ahead, the first ones beside the
// angles: what a block waits for is covered by its own loads and by the SM's other blocks.
// 16384 x 16 heads of 128 bf16: 27 us (0.73 of the copy bandwidth), the gradient 46 us (0.64: two
// sums a head, and 16 running sums of dw a thread leave two blocks an SM); the packed append of 36101
// tokens of 32 + 2 x 8 heads: 169 us (0.77), with the search for a token's row and its page in each block.
// Sums are fp32: of 16 elements in a thread, then over the threads; of dw, over a thread's heads, then
// over threads, warps and blocks, always in the same order.
#include "launch_setup.cuh"
#include "prompt_common.cuh"
#include "rope_common.cuh"

namespace gdnspec {

constexpr int kNormThreads = kRopeThreads;
constexpr int kNormEntries = 8;   // elements or pairs of a head that a lane of its warp takes at most
constexpr int kNormBlocks = 4;    // of an SM: with six the append spills (36101 tokens of 32 + 2 x 8 heads: 226 us, 168 with four)

// Threads that share a head of `units` units of 16 elements: the next power of two.
__host__ __device__ inline int head_lanes(int units) {
    int n = 1;
    while (n < units) n *= 2;
    return n;
}

struct NormArgs {
    const float *weight;   // [D]; null: no norm
    float eps, offset;
};

// Places of unit u's 16 weights in shared memory: four float4, each kind of the units side by side, so that a
// head's threads read neighbouring 16 bytes.
__device__ __forceinline__ int weight_place(int u, int k, int units) { return (k * units + u) * 4; }

// The weights (plus offset) into shared memory, by the block: in the order of the units' runs, or as they are.
template <bool HALF, bool UNITS>
__device__ __forceinline__ void stage_weights(float *ws, const NormArgs &W, const RopeArgs &R) {
    if (!W.weight) return;
    for (int j = threadIdx.x; j < R.D; j += kNormThreads) {
        if (UNITS) {
            const int u = j >> 4, e = j & 15;
            int o0, o1;
            unit_runs<HALF>(u, R.rot, &o0, &o1);
            ws[weight_place(u, e >> 2, R.D >> 4) + (e & 3)] = W.weight[(e < 8 ? o0 : o1) + (e & 7)] + W.offset;
        } else {
            ws[j] = W.weight[j] + W.offset;
        }
    }
}

__device__ __forceinline__ void load_weights(float (&a)[8], float (&b)[8], const float *ws, int u, int units) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 w = *reinterpret_cast<const float4 *>(ws + weight_place(u, k, units));
        float *const z = k < 2 ? a + 4 * k : b + 4 * (k - 2);
        z[0] = w.x, z[1] = w.y, z[2] = w.z, z[3] = w.w;
    }
}

// Head `h` of token `t` of the block's, of the heads that a thread comes to in steps.
struct HeadWalk {
    int t, h, dt, dh, heads;
    __device__ __forceinline__ HeadWalk(int first, int step, int heads_) : heads(heads_) {
        t = first / heads, h = first - t * heads;
        dt = step / heads, dh = step - dt * heads;
    }
    __device__ __forceinline__ void step() {
        t += dt, h += dh;
        if (h >= heads) h -= heads, ++t;
    }
};

// Sum over the `lanes` threads (a power of two, neighbours) of a head; the same in all of them.
__device__ __forceinline__ float head_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float dot16(const float (&a)[8], const float (&b)[8], const float (&c)[8], const float (&d)[8]) {
    float s[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s[i & 1] = fmaf(a[i], c[i], s[i & 1]);
        s[2 + (i & 1)] = fmaf(b[i], d[i], s[2 + (i & 1)]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// The elements of entry e of a head that goes element by element: a pair, or one element behind them (i1 = -1).
template <bool HALF> __device__ __forceinline__ void entry_at(int e, int rot, int *i0, int *i1) {
    const int pairs = rot >> 1;
    *i0 = e < pairs ? (HALF ? e : 2 * e) : pairs + e;
    *i1 = e < pairs ? (HALF ? e + pairs : 2 * e + 1) : -1;
}

// One head by the threads of its warp, element by element: dst = R (r src * w); dst may be src.
template <typename IO, bool HALF>
__device__ __forceinline__ void norm_turn_scalar(const IO *src, IO *dst, const float2 *cs, const float *ws, const NormArgs &W,
                                                 const RopeArgs &R, bool normed, bool turned) {
    const int lane = threadIdx.x & 31, entries = R.D - R.pairs;
    float a[kNormEntries], b[kNormEntries], s = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormEntries; ++i) {
        const int e = lane + 32 * i;
        int i0, i1;
        entry_at<HALF>(e, R.rot, &i0, &i1);
        a[i] = e < entries ? to_f32<IO>(src[i0]) : 0.0f;
        b[i] = e < entries && i1 >= 0 ? to_f32<IO>(src[i1]) : 0.0f;
        s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
    }
    const float r = normed ? rsqrtf(warp_sum(s) / R.D + W.eps) : 1.0f;
#pragma unroll
    for (int i = 0; i < kNormEntries; ++i) {
        const int e = lane + 32 * i;
        if (e >= entries) continue;
        int i0, i1;
        entry_at<HALF>(e, R.rot, &i0, &i1);
        float x = a[i], y = b[i];
        if (normed) {
            x *= r * ws[i0];
            if (i1 >= 0) y *= r * ws[i1];
        }
        if (i1 >= 0) {
            const float c = turned ? cs[e].x : 1.0f, sn = turned ? cs[e].y : 0.0f;
            dst[i0] = from_f32<IO>(turned ? x * c - y * sn : x);
            dst[i1] = from_f32<IO>(turned ? x * sn + y * c : y);
        } else {
            dst[i0] = from_f32<IO>(x);
        }
    }
}

// x and out may be the same memory (a head is read before it is written, by the threads that write it), so neither is
// __restrict__.
template <typename IO, bool HALF, bool UNITS>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
norm_rope_kernel(const __grid_constant__ RopeArgs R, const __grid_constant__ NormArgs W, int N, int heads, int tokens,
                 const int32_t *__restrict__ pos, const IO *x, int64_t x_stride, IO *out, int64_t out_stride) {
    extern __shared__ __align__(16) float2 cs[];   // [tokens][pairs], see turn_place; then the weights
    float *const ws = reinterpret_cast<float *>(cs + tokens * R.pairs + (tokens * R.pairs & 1));
    const int tid = threadIdx.x;
    const int64_t n0 = (int64_t)blockIdx.x * tokens;
    const int live = (int)min((int64_t)tokens, N - n0);
    const int units = R.D >> 4, lanes = head_lanes(units), u = tid & (lanes - 1), turning = R.rot >> 4;
    const float inv_d = 1.0f / R.D;
    int o0 = 0, o1 = 0;
    if (UNITS) unit_runs<HALF>(u, R.rot, &o0, &o1);
    HeadWalk at(tid / lanes, kNormThreads / lanes, heads), ahead = at;
    // A head's elements are loaded while the one before it is worked on, the first ones while cos and sin are formed.  (x and
    // out may be the same memory: those are other heads' places.)
    Run8<IO> r0, r1;
    const auto load = [&] {
        r0.zero();
        r1.zero();
        if (UNITS && ahead.t < live && u < units) {
            const IO *xp = x + (n0 + ahead.t) * x_stride + ahead.h * R.D;
            r0.load(xp + o0);
            r1.load(xp + o1);
        }
        ahead.step();
    };
    grid_dep_wait();
    load();
    stage_weights<HALF, UNITS>(ws, W, R);
    for (int j = tid; j < live * R.pairs; j += kNormThreads) {
        const int t = j / R.pairs, i = j - t * R.pairs;
        cs[t * R.pairs + turn_place<UNITS>(i, R.pairs)] = rope_turn(R, pos[n0 + t], i);
    }
    __syncthreads();
    if (UNITS) {
        // (a warp's threads leave together: the shuffles need them all)
        const int all = live * heads;
        for (int j = (tid & ~31) / lanes; j < all; j += kNormThreads / lanes, at.step()) {
            const bool on = at.t < live && u < units;
            IO *op = out + (n0 + at.t) * out_stride + at.h * R.D;
            float a[8], b[8];
            r0.get(a);
            r1.get(b);
            load();
            const float r = rsqrtf(fmaf(head_sum(dot16(a, b, a, b), lanes), inv_d, W.eps));
            if (!on) continue;
            float wa[8], wb[8];
            load_weights(wa, wb, ws, u, units);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] *= r * wa[i];
                b[i] *= r * wb[i];
            }
            if (u < turning) turn_unit<HALF>(a, b, cs + at.t * R.pairs, u, R.pairs, 1.0f);
            Run8<IO> w0, w1;
            w0.put(a);
            w1.put(b);
            w0.store(op + o0);
            w1.store(op + o1);
        }
    } else {
        for (int j = tid >> 5; j < live * heads; j += kNormThreads / 32) {
            const int t = j / heads, h = j - t * heads;
            norm_turn_scalar<IO, HALF>(x + (n0 + t) * x_stride + h * R.D, out + (n0 + t) * out_stride + h * R.D,
                                       cs + t * R.pairs, ws, W, R, true, true);
        }
    }
}

// Packed prompts: q normed and turned into q_out, k normed and turned and v copied into the pages.  What becomes of a
// token (where its key goes, that it is dead, or that no row owns it) is found by a warp for each token of the block.
template <typename IO, bool HALF, bool UNITS>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
norm_append_kernel(const __grid_constant__ RopeArgs R, const __grid_constant__ NormArgs WQ, const __grid_constant__ NormArgs WK,
                   const __grid_constant__ PromptArgs A, int tokens, const int32_t *__restrict__ pos, const IO *__restrict__ q,
                   int64_t q_stride, const IO *__restrict__ k, int64_t k_stride, const IO *__restrict__ v, int64_t v_stride,
                   IO *__restrict__ q_out) {
    extern __shared__ __align__(16) float2 cs[];   // [tokens][pairs], see turn_place; then both weights
    __shared__ int64_t row_s[kRopeTokens];   // the token's row in the pool; kDead: its q is zero and nothing else is written
    __shared__ int pos_s[kRopeTokens];
    constexpr int64_t kDead = -1, kNobodys = -2, kNoPage = -3;   // (of a page that is none: as kDead, and reported)
    float *const wq = reinterpret_cast<float *>(cs + tokens * R.pairs + (tokens * R.pairs & 1)), *const wk = wq + R.D;
    const KvArgs &C = A.C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n0 = (int64_t)blockIdx.x * tokens;
    const int live = (int)min((int64_t)tokens, A.N - n0);
    const int HQ = A.HQ, heads = HQ + 2 * C.HKV, all = live * heads;
    const int units = R.D >> 4, lanes = head_lanes(units), u = tid & (lanes - 1), turning = R.rot >> 4;
    const float inv_d = 1.0f / R.D;
    int o0 = 0, o1 = 0;
    if (UNITS) unit_runs<HALF>(u, R.rot, &o0, &o1);
    HeadWalk at(tid / lanes, kNormThreads / lanes, heads), ahead = at;
    // A head's elements are loaded while the one before it is worked on, the first ones while the tokens' places and
    // angles are formed (what no row owns is loaded for nothing).
    Run8<IO> x0, x1;
    const auto load = [&] {
        x0.zero();
        x1.zero();
        if (UNITS && ahead.t < live && u < units) {
            const int64_t token = n0 + ahead.t;
            const int h = ahead.h;
            const IO *src = h < HQ ? q + token * q_stride + h * R.D
                          : h < HQ + C.HKV ? k + token * k_stride + (h - HQ) * R.D : v + token * v_stride + (h - HQ - C.HKV) * R.D;
            x0.load(src + o0);
            x1.load(src + o1);
        }
        ahead.step();
    };
    grid_dep_wait();
    load();
    stage_weights<HALF, UNITS>(wq, WQ, R);
    stage_weights<HALF, UNITS>(wk, WK, R);
    const int s0 = tid < A.B ? A.starts[tid] : 0, s1 = tid < A.B ? A.starts[tid + 1] : 0;   // (on their way during what follows)
    uint32_t bits;         // of the rows whose status is this thread's
    const auto look_up = [&](bool all_ascend) {
        bits = 0;
        for (int64_t b = (int64_t)blockIdx.x * kNormThreads + tid; b < A.B; b += (int64_t)gridDim.x * kNormThreads) {
            uint32_t row_bits;
            prompt_row(A, (int)b, all_ascend, &row_bits);
            bits |= row_bits;
        }
        for (int t = warp; t < live; t += kNormThreads / 32) {
            const int token = (int)(n0 + t), b = prompt_owner(A, token, all_ascend);
            if (lane == 0) {
                uint32_t row_bits;
                const PromptRow r = prompt_row(A, b, all_ascend, &row_bits);
                const int at = token - r.first;
                int64_t row = at >= 0 && at < r.owned ? kDead : kNobodys;
                if (at >= 0 && at < r.cnt) {
                    row = kv_token_row(C, r.slot, r.len + at);
                    if (row < 0) row = kNoPage;
                }
                row_s[t] = row;
                pos_s[t] = pos ? pos[token] : r.len + at;
            }
        }
    };
    look_up(true);
    bool ascends = prompt_range(A, s0, s1);   // starts does, as far as the thread sees
    for (int b = tid + kNormThreads; b < A.B; b += kNormThreads) ascends &= prompt_range(A, A.starts[b], A.starts[b + 1]);
    ascends = __syncthreads_and(ascends);
    if (!ascends) {   // the rows that were found need not be the tokens'
        look_up(false);
        __syncthreads();
    }
    if (tid < live && row_s[tid] == kNoPage) bits |= GDN_SPEC_ST_PAGE_OOR;
    if (bits) atomicOr(C.status, bits);
    for (int j = tid; j < live * R.pairs; j += kNormThreads) {
        const int t = j / R.pairs, i = j - t * R.pairs;
        cs[t * R.pairs + turn_place<UNITS>(i, R.pairs)] = rope_turn(R, pos_s[t], i);
    }
    __syncthreads();
    IO *kp = static_cast<IO *>(C.k), *vp = static_cast<IO *>(C.v);
    // where head h of the block's token t goes; null: nowhere
    const auto place = [&](int t, int h) -> IO * {
        const int64_t token = n0 + t, row = row_s[t];
        if (h < HQ) return row == kNobodys ? nullptr : q_out + (token * HQ + h) * R.D;
        if (row < 0) return nullptr;
        return h < HQ + C.HKV ? kp + kv_elem(C, A.layer, h - HQ, row) : vp + kv_elem(C, A.layer, h - HQ - C.HKV, row);
    };
    if (UNITS) {
        for (int j = (tid & ~31) / lanes; j < all; j += kNormThreads / lanes, at.step()) {
            const int t = at.t, h = at.h;
            IO *const dst = t < live && u < units ? place(t, h) : nullptr;
            const bool is_q = h < HQ, is_v = h >= HQ + C.HKV;
            float a[8], b[8];
            Run8<IO> r0 = x0, r1 = x1;
            load();
            r0.get(a);
            r1.get(b);
            const float r = rsqrtf(fmaf(head_sum(dot16(a, b, a, b), lanes), inv_d, is_q ? WQ.eps : WK.eps));
            if (!dst) continue;
            if (row_s[t] < 0) {
                r0.zero();
                r1.zero();
            } else if (!is_v) {
                if (is_q ? WQ.weight != nullptr : WK.weight != nullptr) {
                    float wa[8], wb[8];
                    load_weights(wa, wb, is_q ? wq : wk, u, units);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] *= r * wa[i];
                        b[i] *= r * wb[i];
                    }
                }
                if (u < turning) turn_unit<HALF>(a, b, cs + t * R.pairs, u, R.pairs, 1.0f);
                r0.put(a);
                r1.put(b);
            }
            r0.store(dst + o0);
            r1.store(dst + o1);
        }
    } else {
        for (int j = warp; j < all; j += kNormThreads / 32) {
            const int t = j / heads, h = j - t * heads;
            const int64_t token = n0 + t;
            IO *const dst = place(t, h);
            if (!dst) continue;
            const IO *src = h < HQ ? q + token * q_stride + h * R.D
                          : h < HQ + C.HKV ? k + token * k_stride + (h - HQ) * R.D : v + token * v_stride + (h - HQ - C.HKV) * R.D;
            if (row_s[t] < 0 || h >= HQ + C.HKV) {
                for (int d = lane; d < R.D; d += 32) dst[d] = row_s[t] < 0 ? from_f32<IO>(0.0f) : src[d];
                continue;
            }
            const NormArgs &W = h < HQ ? WQ : WK;
            norm_turn_scalar<IO, HALF>(src, dst, cs + t * R.pairs, h < HQ ? wq : wk, W, R, W.weight != nullptr, true);
        }
    }
}

// ------------------------------------------------------------------ gradient

// dx may be x or dy itself, as above.  A thread takes the same elements of every head that it comes to, so its part of dw
// stays in registers; a block's is put together in shared memory and kept in `part` [blocks][D]
// for the kernel that sums the blocks' (one block: it is dw).
template <typename IO, bool HALF, bool UNITS>
__global__ void __launch_bounds__(kNormThreads, 2)
norm_grad_kernel(const __grid_constant__ RopeArgs R, const __grid_constant__ NormArgs W, int N, int heads, int tokens,
                 const int32_t *__restrict__ pos, const IO *x, int64_t x_stride, const IO *dy, int64_t dy_stride, IO *dx,
                 int64_t dx_stride, float *part) {
    extern __shared__ __align__(16) float2 cs[];   // [tokens][pairs], see turn_place; then the weights; then [8][D] sums
    float *const ws = reinterpret_cast<float *>(cs + tokens * R.pairs + (tokens * R.pairs & 1)), *const sums = ws + R.D;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = R.D >> 4, lanes = UNITS ? head_lanes(units) : 32, u = tid & (lanes - 1), turning = R.rot >> 4;
    int o0 = 0, o1 = 0;
    if (UNITS) unit_runs<HALF>(u, R.rot, &o0, &o1);
    float da[8] = {}, db[8] = {};   // of the unit's two runs, or of the lane's entries
    const float inv_d = 1.0f / R.D;
    const HeadWalk first(tid / lanes, kNormThreads / lanes, heads);
    Run8<IO> x0, x1, y0, y1;        // the next head's elements, of x and of dy
    const auto load = [&](int64_t n0, HeadWalk &ahead) {
        x0.zero();
        x1.zero();
        y0.zero();
        y1.zero();
        if (ahead.t < tokens && n0 + ahead.t < N && u < units) {
            const IO *xp = x + (n0 + ahead.t) * x_stride + ahead.h * R.D, *yp = dy + (n0 + ahead.t) * dy_stride + ahead.h * R.D;
            x0.load(xp + o0);
            x1.load(xp + o1);
            y0.load(yp + o0);
            y1.load(yp + o1);
        }
        ahead.step();
    };
    grid_dep_wait();
    stage_weights<HALF, UNITS>(ws, W, R);
    for (int64_t n0 = (int64_t)blockIdx.x * tokens; n0 < N; n0 += (int64_t)gridDim.x * tokens) {
        const int live = (int)min((int64_t)tokens, N - n0), all = live * heads;
        HeadWalk at = first, ahead = first;
        if (UNITS) load(n0, ahead);
        __syncthreads();   // the tokens before are done with their cos and sin
        for (int j = tid; j < live * R.pairs; j += kNormThreads) {
            const int t = j / R.pairs, i = j - t * R.pairs;
            cs[t * R.pairs + turn_place<UNITS>(i, R.pairs)] = rope_turn(R, pos[n0 + t], i);
        }
        __syncthreads();
        for (int j = (tid & ~31) / lanes; j < all; j += kNormThreads / lanes, at.step()) {
            const int t = at.t, h = at.h;
            const IO *xp = x + (n0 + t) * x_stride + h * R.D, *yp = dy + (n0 + t) * dy_stride + h * R.D;
            IO *op = dx + (n0 + t) * dx_stride + h * R.D;
            if (UNITS) {
                const bool on = t < live && u < units;
                float a[8], b[8], ga[8], gb[8], wa[8] = {}, wb[8] = {};
                x0.get(a);
                x1.get(b);
                y0.get(ga);
                y1.get(gb);
                load(n0, ahead);
                if (on) {
                    if (u < turning) turn_unit<HALF>(ga, gb, cs + t * R.pairs, u, R.pairs, -1.0f);
                    load_weights(wa, wb, ws, u, units);
                }
                const float r = rsqrtf(fmaf(head_sum(dot16(a, b, a, b), lanes), inv_d, W.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    da[i] = fmaf(r * a[i], ga[i], da[i]);
                    db[i] = fmaf(r * b[i], gb[i], db[i]);
                    ga[i] *= wa[i];
                    gb[i] *= wb[i];
                }
                const float c = r * r * (head_sum(dot16(a, b, ga, gb), lanes) * inv_d);
                if (!on) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = r * (ga[i] - c * a[i]);
                    b[i] = r * (gb[i] - c * b[i]);
                }
                Run8<IO> r0, r1;
                r0.put(a);
                r1.put(b);
                r0.store(op + o0);
                r1.store(op + o1);
            } else {
                const int entries = R.D - R.pairs;
                float a[kNormEntries], b[kNormEntries], ga[kNormEntries], gb[kNormEntries], s = 0.0f, sg = 0.0f;
#pragma unroll
                for (int i = 0; i < kNormEntries; ++i) {
                    const int e = lane + 32 * i;
                    int i0, i1;
                    entry_at<HALF>(e, R.rot, &i0, &i1);
                    const bool one = e < entries, two = one && i1 >= 0;
                    a[i] = one ? to_f32<IO>(xp[i0]) : 0.0f;
                    b[i] = two ? to_f32<IO>(xp[i1]) : 0.0f;
                    const float g = one ? to_f32<IO>(yp[i0]) : 0.0f, f = two ? to_f32<IO>(yp[i1]) : 0.0f;
                    const float2 turn = two ? cs[t * R.pairs + e] : make_float2(1.0f, 0.0f);
                    ga[i] = two ? g * turn.x + f * turn.y : g;
                    gb[i] = two ? f * turn.x - g * turn.y : 0.0f;
                    s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
                }
                const float r = rsqrtf(warp_sum(s) / R.D + W.eps);
#pragma unroll
                for (int i = 0; i < kNormEntries; ++i) {
                    const int e = lane + 32 * i;
                    int i0, i1;
                    entry_at<HALF>(e, R.rot, &i0, &i1);
                    da[i] = fmaf(r * a[i], ga[i], da[i]);
                    db[i] = fmaf(r * b[i], gb[i], db[i]);
                    ga[i] *= e < entries ? ws[i0] : 0.0f;
                    gb[i] *= e < entries && i1 >= 0 ? ws[i1] : 0.0f;
                    sg = fmaf(a[i], ga[i], fmaf(b[i], gb[i], sg));
                }
                const float c = r * r * (warp_sum(sg) / R.D);
#pragma unroll
                for (int i = 0; i < kNormEntries; ++i) {
                    const int e = lane + 32 * i;
                    if (e >= entries) continue;
                    int i0, i1;
                    entry_at<HALF>(e, R.rot, &i0, &i1);
                    op[i0] = from_f32<IO>(r * (ga[i] - c * a[i]));
                    if (i1 >= 0) op[i1] = from_f32<IO>(r * (gb[i] - c * b[i]));
                }
            }
        }
    }
    __syncthreads();
    if (UNITS) {   // over the heads of a warp, then over the warps
#pragma unroll
        for (int i = 0; i < 8; ++i)
            for (int o = lanes; o < 32; o <<= 1) {
                da[i] += __shfl_xor_sync(0xffffffffu, da[i], o);
                db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
            }
        if (lane < units) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[warp * R.D + o0 + i] = da[i];
                sums[warp * R.D + o1 + i] = db[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNormEntries; ++i) {
            const int e = lane + 32 * i;
            if (e >= R.D - R.pairs) continue;
            int i0, i1;
            entry_at<HALF>(e, R.rot, &i0, &i1);
            sums[warp * R.D + i0] = da[i];
            if (i1 >= 0) sums[warp * R.D + i1] = db[i];
        }
    }
    __syncthreads();
    for (int d = tid; d < R.D; d += kNormThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kNormThreads / 32; ++w) s += sums[w * R.D + d];
        part[(int64_t)blockIdx.x * R.D + d] = s;
    }
    grid_dep_launch();
}

// dw = the sum of the blocks' parts, always in the same order: 32 columns a block, a row of parts a warp in turn.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float *__restrict__ part, int blocks, int D, float *dw) {
    __shared__ float s_s[kSumThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    grid_dep_wait();
    float s = 0.0f;
#pragma unroll 8
    for (int b = warp; b < blocks; b += kSumThreads / 32)
        if (d < D) s += part[(int64_t)b * D + d];
    s_s[warp][lane] = s;
    __syncthreads();
    const float t = warp_sum(s_s[lane][warp]);   // column `warp`
    if (lane == 0 && blockIdx.x * 32 + warp < D) dw[blockIdx.x * 32 + warp] = t;
    grid_dep_launch();
}

// ------------------------------------------------------------------ launch

// Tokens of a block: four once that still gives every SM several blocks, and more while they have few units of 16 elements.
static int norm_tokens(int64_t n, int units) {
    int t = n >= 4096 ? 4 : 1;
    while (t >= 4 && t < kRopeTokens && t * units < 8 * kNormThreads && n >= 4096 * t) t *= 2;
    return t;
}

// Shared memory of `tokens` tokens' cos and sin and `weights` rows of D floats.
static size_t norm_smem(const RopeArgs &R, int tokens, int weights) {
    const int turns = tokens * R.pairs;
    return (turns + (turns & 1)) * sizeof(float2) + (size_t)weights * R.D * sizeof(float);
}

static NormArgs norm_args(const gdn_spec_head_norm *n) { return n ? NormArgs{n->weight, n->eps, n->offset} : NormArgs{nullptr, 1.0f, 0.0f}; }

template <typename IO, bool HALF, bool UNITS>
static cudaError_t run_norm(const RopeArgs &R, const NormArgs &W, int N, int heads, const int32_t *pos, const void *x,
                            int64_t x_stride, void *out, int64_t out_stride, cudaStream_t st) {
    const int tokens = norm_tokens(N, heads * R.D / 16);
    const int64_t blocks = ((int64_t)N + tokens - 1) / tokens;
    return launch_dependent(norm_rope_kernel<IO, HALF, UNITS>, dim3((unsigned)blocks), dim3(kNormThreads), norm_smem(R, tokens, 1),
                            st, R, W, N, heads, tokens, pos, static_cast<const IO *>(x), x_stride, static_cast<IO *>(out), out_stride);
}

// The kernel of a type, a layout and whether heads come in units of 16.
#define GDN_SPEC_ROPE_KERNEL(run, bf16, half, units)                                                                   \
    ((bf16) ? ((units) ? ((half) ? run<__nv_bfloat16, true, true> : run<__nv_bfloat16, false, true>)                   \
                       : ((half) ? run<__nv_bfloat16, true, false> : run<__nv_bfloat16, false, false>))                \
            : ((units) ? ((half) ? run<float, true, true> : run<float, false, true>)                                   \
                       : ((half) ? run<float, true, false> : run<float, false, false>)))

static bool in_units(const gdn_spec_rope_plan *p) { return p->D % 16 == 0 && p->rot % 16 == 0; }

cudaError_t launch_norm_rope(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *norm, int N, int heads, bool bf16,
                             const int32_t *pos, const void *x, int64_t x_stride, void *out, int64_t out_stride, cudaStream_t st) {
    const auto go = GDN_SPEC_ROPE_KERNEL(run_norm, bf16, plan->layout == GDN_SPEC_ROPE_HALF, in_units(plan));
    return go(rope_args(plan), norm_args(norm), N, heads, pos, x, x_stride, out, out_stride, st);
}

template <typename IO, bool HALF, bool UNITS>
static cudaError_t run_norm_append(const RopeArgs &R, const NormArgs &WQ, const NormArgs &WK, const PromptArgs &A,
                                   const int32_t *pos, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                   const void *v, int64_t v_stride, cudaStream_t st) {
    const int tokens = norm_tokens(A.N, (A.HQ + 2 * A.C.HKV) * R.D / 16);
    return launch_dependent(norm_append_kernel<IO, HALF, UNITS>, dim3((unsigned)(((int64_t)A.N + tokens - 1) / tokens)),
                            dim3(kNormThreads), norm_smem(R, tokens, 2), st, R, WQ, WK, A, tokens, pos,
                            static_cast<const IO *>(q), q_stride, static_cast<const IO *>(k), k_stride,
                            static_cast<const IO *>(v), v_stride, static_cast<IO *>(A.out));
}

// A: the cache, layer, rows and packed tokens; out is q_out.
cudaError_t launch_norm_rope_append(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *q_norm, const gdn_spec_head_norm *k_norm,
                                    const PromptArgs &A, bool bf16, const int32_t *pos, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v, int64_t v_stride, cudaStream_t st) {
    const auto go = GDN_SPEC_ROPE_KERNEL(run_norm_append, bf16, plan->layout == GDN_SPEC_ROPE_HALF, in_units(plan));
    return go(rope_args(plan), norm_args(q_norm), norm_args(k_norm), A, pos, q, q_stride, k, k_stride, v, v_stride, st);
}

// Tokens that a block of the gradient takes at a time, and blocks: a resident grid, or fewer where the tokens are fewer.
static int grad_tokens(int N, int heads) {
    int t = 1;
    while (t < kRopeTokens && t * heads < 128 && N >= 1024 * t) t *= 2;
    return t;
}
int norm_grad_blocks(int N, int heads, int sms) {
    const int64_t need = ((int64_t)N + grad_tokens(N, heads) - 1) / grad_tokens(N, heads);
    return (int)(need < 2 * sms ? need : 2 * sms);
}

template <typename IO, bool HALF, bool UNITS>
static cudaError_t run_norm_grad(const RopeArgs &R, const NormArgs &W, int N, int heads, int blocks, const int32_t *pos,
                                 const void *x, int64_t x_stride, const void *dy, int64_t dy_stride, void *dx, int64_t dx_stride,
                                 float *part, cudaStream_t st) {
    const int tokens = grad_tokens(N, heads);
    return launch_dependent(norm_grad_kernel<IO, HALF, UNITS>, dim3(blocks), dim3(kNormThreads),
                            norm_smem(R, tokens, 1 + kNormThreads / 32), st, R, W, N, heads, tokens, pos, static_cast<const IO *>(x),
                            x_stride, static_cast<const IO *>(dy), dy_stride, static_cast<IO *>(dx), dx_stride, part);
}

cudaError_t launch_norm_rope_grad(const gdn_spec_rope_plan *plan, const gdn_spec_head_norm *norm, int N, int heads, bool bf16,
                                  int sms, const int32_t *pos, const void *x, int64_t x_stride, const void *dy, int64_t dy_stride,
                                  void *dx, int64_t dx_stride, float *dw, float *part, cudaStream_t st) {
    const int blocks = norm_grad_blocks(N, heads, sms);
    const auto go = GDN_SPEC_ROPE_KERNEL(run_norm_grad, bf16, plan->layout == GDN_SPEC_ROPE_HALF, in_units(plan));
    const cudaError_t e = go(rope_args(plan), norm_args(norm), N, heads, blocks, pos, x, x_stride, dy, dy_stride, dx, dx_stride,
                             blocks == 1 ? dw : part, st);
    if (e != cudaSuccess || blocks == 1) return e;
    return launch_dependent(norm_sum_kernel, dim3((plan->D + 31) / 32), dim3(kSumThreads), 0, st, (const float *)part, blocks, (int)plan->D, dw);
}

}  // namespace gdnspec
