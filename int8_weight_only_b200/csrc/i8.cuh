// Device helpers of the int8-activation operators alone: wait sites, pairs of
// fp32, the 8-bit integer tensor-core product and its operands.  They stand
// apart from common.cuh so that the code of the W8A16 kernels, and with it
// their committed ncu captures, stays as captured when these change.
#pragma once

#include "common.cuh"

namespace w8 {

// Wait sites, beside those of WaitSite.
enum I8WaitSite : unsigned {
    SITE_I8_EMPTY = 0x60,
    SITE_I8_FULL = 0x61,
    SITE_I8_DEMPTY = 0x62,
    SITE_I8_DFULL = 0x63,
    SITE_I8_DRAIN = 0x64,
};

// ---------------------------------------------------------------- pairs of fp32
// Two IEEE operations in one instruction.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_sub(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---------------------------------------------------------------- tcgen05
// As smem_desc_kmajor_sw128, for a tile with 64-byte swizzle (the packed weight
// tile: rows of 64 bytes, 16-byte chunk c of row r at slot c XOR ((r >> 1) & 3)):
// 8-row groups 512 bytes apart, layout type 4.
__device__ __forceinline__ uint64_t smem_desc_kmajor_sw64(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)(512u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)4u << 61;
    return d;
}

// One lane of a converged warp.  A branch on this, unlike one on the lane
// number, keeps the operands of the instructions under it warp-uniform.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[smem desc] * B[smem desc], kind::i8 (8-bit integers, 32-bit
// integer accumulator), K = 32.
__device__ __forceinline__ void tc_mma_ss_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same on a pair of SMs (cta_group::2).
__device__ __forceinline__ void tc_mma_ss_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor for kind::i8: A unsigned 8-bit (a_format, bits 7-9,
// 0), B signed 8-bit (b_format, bits 10-12, 1), 32-bit integer accumulator
// (c_format, bits 4-5, 2) without saturation (bit 3), both operands K-major,
// shape M x N.
__host__ __device__ constexpr uint32_t idesc_u8_s8_s32(uint32_t m, uint32_t n) {
    return (2u << 4) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Load 16 columns of this warp's 32 lanes and wait for them, in one asm
// statement (see tmem_load_32).
__device__ __forceinline__ void tmem_load_16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// Load 32 columns of 16 tensor-memory lanes, in the order of 16 x 8 fragments
// (four column groups i of 8 columns, registers 4 i ...): register 4 i + j of
// thread t holds lane t / 4 + 8 (j / 2), column 8 i + 2 (t % 4) + j % 2.  One
// statement with its wait (see tmem_load_32).
__device__ __forceinline__ void tmem_load_frag_16x32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// Store four 8 x 8 matrices of 16-bit values transposed: register i holds
// matrix i as the product's fragments do (thread t: row t / 4, columns
// 2 (t % 4) and + 1); its columns become rows of 16 bytes at the addresses
// that threads 8 i ... 8 i + 7 give.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t smem_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

}  // namespace w8
