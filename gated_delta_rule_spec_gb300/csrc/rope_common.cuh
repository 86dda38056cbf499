// rope_common.cuh -- what the kernels of rotary positions share: the angle of a pair,
// eight elements at a time, and how a head is cut into units of sixteen elements.
//
// Pair i of a head is turned by the angle pos * f_i.  The plan holds f_i as a
// fraction of 2^64 of a turn, so pos * freq modulo 2^64 is the angle modulo a
// turn, exact to 2^-64 pos.
#pragma once

#include "kv_common.cuh"

namespace gdnspec {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeTokens = 16;   // tokens of a block at most

struct RopeArgs {
    int D, rot, pairs;
    float mscale;
    uint64_t freq[kRopeMaxPairs];
};

// cos and sin of pair i at position pos, times mscale
__device__ __forceinline__ float2 rope_turn(const RopeArgs &R, int pos, int i) {
    const uint64_t turn = (uint64_t)(int64_t)pos * R.freq[i];
    // the signed fraction in half turns, [-1, 1)
    const float half_turns = __ll2float_rn((int64_t)turn) * 0x1p-63f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * R.mscale, s * R.mscale);
}

// Eight consecutive elements in 32 bits.
template <typename IO> struct Run8;
template <> struct Run8<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
};
template <> struct Run8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};

// Where pair i's cos and sin stand among a token's: units of eight pairs are spread so that a warp's lanes, which turn
// neighbouring units, read neighbouring 16 bytes (two pairs).
template <bool UNITS> __device__ __forceinline__ int turn_place(int i, int pairs) {
    return UNITS ? ((i & 7) >> 1) * (pairs >> 2) + (i >> 3) * 2 + (i & 1) : i;
}

// One unit of a head: the two runs at offsets o0 and o1, turned by the pairs
// of unit u (interleaved: run 0 holds its first four pairs, run 1 the others;
// half: all of them across the runs).
template <bool HALF>
__device__ __forceinline__ void turn_unit(float (&x)[8], float (&y)[8], const float2 *cs, int u, int pairs, float sign) {
    const auto turn = [sign](float &a, float &b, float c, float s) {
        s *= sign;
        const float a0 = a, b0 = b;
        a = a0 * c - b0 * s;
        b = a0 * s + b0 * c;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 t = *reinterpret_cast<const float4 *>(cs + k * (pairs >> 2) + u * 2);
        if (HALF) {
            turn(x[2 * k], y[2 * k], t.x, t.y);
            turn(x[2 * k + 1], y[2 * k + 1], t.z, t.w);
        } else {
            float *const z = k < 2 ? x + 4 * k : y + 4 * (k - 2);
            turn(z[0], z[1], t.x, t.y);
            turn(z[2], z[3], t.z, t.w);
        }
    }
}
template <typename IO, bool HALF>
__device__ __forceinline__ void turn_unit(Run8<IO> &r0, Run8<IO> &r1, const float2 *cs, int u, int pairs, float sign) {
    float x[8], y[8];
    r0.get(x);
    r1.get(y);
    turn_unit<HALF>(x, y, cs, u, pairs, sign);
    r0.put(x);
    r1.put(y);
}

// How a head is cut into units of 16 elements: rot / 16 that turn, then the rest
// (D and rot multiples of 16; other dims go element by element: 32768 tokens of 32 heads
// of 96 dims, 24 of them turned, take 317 us in bf16, and 62 with 32 turned).
template <bool HALF>
__device__ __forceinline__ void unit_runs(int u, int rot, int *o0, int *o1) {
    const bool turn = u < (rot >> 4);
    *o0 = HALF && turn ? u * 8 : u * 16;
    *o1 = HALF && turn ? (rot >> 1) + u * 8 : u * 16 + 8;
}

// One element of a turned head, for dims that do not come in units of 16.
template <typename IO, bool HALF>
__device__ __forceinline__ void turn_scalar(const IO *x, IO *y, const float2 *cs, int rot, int D, float sign, int e) {
    // e < rot / 2: pair e; else the element rot + e - rot / 2
    const int pairs = rot >> 1;
    if (e < pairs) {
        const int i0 = HALF ? e : 2 * e, i1 = HALF ? e + pairs : 2 * e + 1;
        const float c = cs[e].x, s = cs[e].y * sign, a = to_f32<IO>(x[i0]), b = to_f32<IO>(x[i1]);
        y[i0] = from_f32<IO>(a * c - b * s);
        y[i1] = from_f32<IO>(a * s + b * c);
    } else {
        const int i = rot + e - pairs;
        y[i] = x[i];
    }
}

inline RopeArgs rope_args(const gdn_spec_rope_plan *p) {
    RopeArgs R;
    R.D = p->D;
    R.rot = p->rot;
    R.pairs = p->rot / 2;
    R.mscale = p->mscale;
    for (int i = 0; i < kRopeMaxPairs; ++i) R.freq[i] = i < R.pairs ? p->freq[i] : 0;
    return R;
}

}  // namespace gdnspec
