// attn_tc.cuh -- what the tensor-core attention kernels share: bounded waits of whole
// warps, uniform operands, packed fp32 arithmetic for the softmax, and the encoding
// of their tensor maps.
#pragma once

#include <mutex>

#include <cuda.h>

#include "ptx_attn.cuh"

namespace gdnspec {
namespace tat {

constexpr float kGrow = 8.0f;            // log2 of what the maximum may grow by before it is moved
constexpr uint32_t kPolls = 1u << 18;    // of a wait, before it gives up (half a second)

// Bounded wait of a whole warp, which also ends when another role has given up; one
// answer for all lanes.  It looks first: a phase that has passed costs some 50 cycles so,
// and 260 by a poll.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t limit = kPolls) {
    bool ok = false;
    if (limit) ok = ptx::mbar_test_wait(bar, parity);
#pragma unroll 1
    for (uint32_t it = 0; !ok && it < limit; ++it) {
        ok = ptx::mbar_try_wait(bar, parity);
        if (!ok && (it & 15u) == 15u && *abort) break;
    }
    if (!ok) *abort = 1;
    return __all_sync(0xffffffffu, ok);
}

// A value that all lanes hold, from one of them: the tensor core's operands are uniform
// registers, and values that come from memory or from a loop are only seen to be
// uniform behind a shuffle (without it each MMA costs some 300 cycles to issue).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Place in a ring of `size` stages.
struct Place {
    uint32_t at = 0, ph = 0;
    __device__ __forceinline__ void step(uint32_t size) {
        if (++at == size) {
            at = 0;
            ph ^= 1u;
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a tcgen05.ld brought is only valid behind its wait: uses depend on this.
template <int N>
__device__ __forceinline__ void landed(uint32_t (&r)[N]) {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void commit(uint32_t bar) {
    if (ptx::elect_one()) ptx::mma_commit(bar);
    __syncwarp();
}

// ------------------------------------------------------------------ host

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// bf16 tensor of `rank` dims, the innermost `dims[0]` dense; strides in elements.
inline bool bf16_map(CUtensorMap *map, const void *p, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                     const cuuint32_t *box) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t bytes[3];
    cuuint32_t one[3] = {1, 1, 1};
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] * 2;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(p), dims, bytes, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tat
}  // namespace gdnspec
