// Warp-wide matrix products for work of too few rows for tcgen05 tiles, copies by
// thread into shared memory, and numbers as two bf16 parts.
//
// Fragments of mma.m16n8k16, with g = lane / 4 and c = lane % 4: A holds rows g
// and g + 8 at columns 2c, 2c + 1 (registers 0, 1) and 8 further (2, 3), B rows
// 2c, 2c + 1 and 8 further of column g, the sums rows g and g + 8 of columns 2c,
// 2c + 1.
#pragma once
#include "common.cuh"

namespace bss {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;       // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// An 8 x 8 block of 16-bit elements transposed: from (row g, columns 2c, 2c + 1)
// to (column g, rows 2c, 2c + 1).
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// fp16 operands (F16) or bf16 ones, fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A number as two bf16 ones, its high half cut off and the rest, of which bf16
// holds all but 2^-15 of the number: the high halves of two, packed, and a rest.
__device__ __forceinline__ uint32_t high_bf16(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float low_part(float x) {
  return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
}

}  // namespace bss
