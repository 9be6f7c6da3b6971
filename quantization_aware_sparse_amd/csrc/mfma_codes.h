// Codes as operands of the bf16 matrix instruction v_mfma_f32_16x16x32_bf16.
#pragma once

#include "common.h"

namespace qwha {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// (x & mask) | bits in one instruction, where the mask is in a vector register
// (one scalar operand per instruction). Left to the compiler: it knows the wait
// states between the instruction's result and a matrix instruction that reads it.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  return (x & mask) | bits;
}
__device__ __forceinline__ uint32_t in_vgpr(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ bf16x8 as_operand(const uint32_t* d) {
  bf16x8 r;
  __builtin_memcpy(&r, d, 16);
  return r;
}

// 8 4-bit codes of a word as bf16(16 + q) = 0x4180 | q << 3: low nibbles from
// w << 3, high ones from w >> 1, a byte of each to a pair. `mask` is
// kMask4 in a vector register.
constexpr uint32_t kMask4 = 0x00780078u;
constexpr uint32_t kBase4 = 0x41804180u;
__device__ __forceinline__ bf16x8 operand4(uint32_t w, uint32_t mask) {
  const uint32_t lo = w << 3, hi = w >> 1;
  uint32_t d[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    d[k] = and_or(__builtin_amdgcn_perm(hi, lo, 0x0C040C00u + 0x00010001u * k), mask, kBase4);
  return as_operand(d);
}

// byte k of w as fp32 (a small integer: its upper half is the bf16)
__device__ __forceinline__ uint32_t byte_f32(uint32_t w, int k) {
  return __float_as_uint(static_cast<float>((w >> (8 * k)) & 0xFFu));
}
// 8 8-bit codes of two words as bf16(q)
__device__ __forceinline__ bf16x8 operand8(uint32_t w0, uint32_t w1) {
  uint32_t d[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k < 2 ? w0 : w1;
    d[k] = __builtin_amdgcn_perm(byte_f32(w, 2 * (k % 2) + 1), byte_f32(w, 2 * (k % 2)),
                                 0x07060302u);
  }
  return as_operand(d);
}

}  // namespace qwha
