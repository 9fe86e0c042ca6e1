// Inline-PTX wrappers the attention kernels need beside ptx.cuh: 32-column
// TMEM loads and stores, MMAs with the A operand in TMEM, descriptors of
// operands whose rows run along M or N, packed fp32 arithmetic and base-2
// exponentials.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace convgb300 {

// 32 lanes x 32 columns of 32 bits (see tmem_ld_32x32b_x16).
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// 16 columns of an array's part.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* v) {
  tmem_ld_32x32b_x16(taddr, *reinterpret_cast<uint32_t(*)[16]>(v));
}
__device__ __forceinline__ void tmem_wait_ld_x16(uint32_t* v) {
  tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[16]>(v));
}

// tcgen05.wait::ld naming the registers of an earlier 32-column load, so that
// no use of them moves above the wait.
__device__ __forceinline__ void tmem_wait_ld_x32(uint32_t* v) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
        "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
        "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]),
        "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
        "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
      :
      : "memory");
}

// After a tcgen05.wait::ld: names n registers (a multiple of 8) of an earlier
// load, so that no use of them moves above the wait.  No instruction.  (Each
// wait costs tens of cycles even when there is nothing to wait for: loads
// share one.)
template <int n>
__device__ __forceinline__ void tmem_pin(uint32_t* v) {
#pragma unroll
  for (int i = 0; i < n; i += 8)
    asm volatile(""
                 : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]),
                   "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptors of 128-byte-swizzled operands.  The high
// word is the same for all: 8-row groups 1024 bytes apart (stride offset),
// descriptor version, layout.  The low word holds the address >> 4 and the
// leading offset >> 4: unused for operands whose 128-byte rows run along K
// (K-major); for rows that run along M or N (64 elements, one row per K), the
// distance of blocks of 64 M or N.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
constexpr uint32_t kLeadK = 1u << 16;
__device__ __forceinline__ uint32_t lead_mn(uint32_t block_bytes) { return (block_bytes >> 4) << 16; }

// Up to four consecutive K-steps (16 elements each) of D[tmem] (+)= A[smem]
// B[smem]^T, both K-major: one elected lane issues them back to back.  Every
// lane of the warp runs this with the same operands.  (One MMA per call, with
// its descriptors built in C++, cost about 100 cycles of issue each, twice
// what the tensor core takes for a 128x128x16 step.)
// A step moves A by kA and B by kB units of 16 bytes: 2 along K (K-major),
// 128 down 16 rows (rows along M or N).
template <int kA, int kB>
__device__ __forceinline__ void mma_x4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate, int steps) {
  asm volatile(
      "{\n\t.reg .pred e, p, t, q;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
      "setp.gt.and.s32 q, %6, 1, e;\n\t"
      "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "setp.gt.and.s32 q, %6, 2, e;\n\t"
      "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "setp.gt.and.s32 q, %6, 3, e;\n\t"
      "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHigh), "r"(idesc), "r"(accumulate), "r"(steps), "n"(kA), "n"(kB)
      : "memory");
}
__device__ __forceinline__ void mma_ss_x4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate, int steps) {
  mma_x4<2, 2>(d, a_lo, b_lo, idesc, accumulate, steps);
}

// The same with A in TMEM (two K elements per 32-bit column, 8 columns a step;
// the second step begins kSecond columns on, the third kThird) and B's rows
// running along N (a step is 16 rows of 128 bytes).
template <int kThird = 16, int kSecond = 8>
__device__ __forceinline__ void mma_ts_x4(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate, int steps) {
  asm volatile(
      "{\n\t.reg .pred e, p, t, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t"
      "setp.gt.and.s32 q, %6, 1, e;\n\t"
      "add.s32 a, %1, %9;\n\tadd.s64 b, b, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "setp.gt.and.s32 q, %6, 2, e;\n\t"
      "add.s32 a, %1, %7;\n\tadd.s64 b, b, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "setp.gt.and.s32 q, %6, 3, e;\n\t"
      "add.s32 a, %1, %8;\n\tadd.s64 b, b, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHigh), "r"(idesc), "r"(accumulate), "r"(steps), "n"(kThird),
      "n"(kThird + kSecond), "n"(kSecond)
      : "memory");
}

// kind::f16 instruction descriptor: fp32 accumulators, both operands of one
// 16-bit type (see make_idesc), M = 128; operands along M or N flagged.
__host__ __device__ constexpr uint32_t attn_idesc(bool bf16, uint32_t n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Moves registers between the warpgroups of a block: the sum over the block's
// warpgroups stays within what it was launched with.
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace convgb300
