// ptx_attn.cuh -- more inline-PTX wrappers, for the tree attention's kernel: an
// arrive and a poll of an mbarrier, TMEM moves of raw bits, the MN-major operand
// descriptor, the bf16 MMA with A in tensor memory, and the elected lane.
#pragma once

#include "ptx_sm100.cuh"

namespace gdnspec {
namespace ptx {

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One poll of phase `parity` that may be suspended for a time of the machine's
// choosing (some microseconds at most, as measured); it resumes sooner after the
// phase completes than the poll with a hint (a round trip between two warps
// takes 219 cycles against 281).
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P1;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Warp-wide: true in one lane, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Shared-memory matrix descriptor: MN-major operand in the 128-byte swizzle
// layout (a row holds 64 consecutive 16-bit elements of the M or N dimension for one
// index of the contraction; 8 such rows form a 1024-byte group, groups of the
// contraction follow each other, and the next 64 elements of M or N are `mn_stride`
// bytes away).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t addr, uint32_t mn_stride) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);             // start address
    d |= (uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16;  // leading byte offset: next 64 elements
    d |= (uint64_t)(1024u >> 4) << 32;                  // stride byte offset: next 8 of the contraction
    d |= (uint64_t)1u << 46;                            // descriptor version (sm_100 family)
    d |= (uint64_t)2u << 61;                            // layout: 128-byte swizzle
    return d;
}

// Bit of the instruction descriptor that makes B MN-major.
constexpr uint32_t kIdescBMn = 1u << 16;

// D[tmem] (+)= A[tmem] * B[smem], one MMA of K = 16 bf16 elements; A is M lanes x 8
// consecutive 32-bit columns of tensor memory, two elements a column.
__device__ __forceinline__ void mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Warp-wide: 32 consecutive 32-bit TMEM columns of this thread's lane, as bits
// (valid after tmem_ld_wait).
__device__ __forceinline__ void tmem_ld32_bits(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Warp-wide: store 16 consecutive 32-bit TMEM columns of this thread's lane, as bits.
__device__ __forceinline__ void tmem_st16_bits(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 "
        "[%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

}  // namespace ptx
}  // namespace gdnspec
