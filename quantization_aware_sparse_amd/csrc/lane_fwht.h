// The Walsh-Hadamard transform of rows that lie across the lanes of a wave:
// out[j] = sum_m in[m] * (-1)^popcount(m & j), N = 64, 128 or 256 columns.
#pragma once

#include "common.h"

namespace qwha {

// lane ^ X's values added, or the lane's own subtracted from them
template <int X, int PER, typename Acc>
__device__ __forceinline__ void butterfly_lanes(Acc* v, int lane) {
  const Acc sign = lane & X ? Acc(-1) : Acc(1);
#pragma unroll
  for (int r = 0; r < PER; ++r) v[r] = lane_xor<X>(v[r]) + sign * v[r];
}

// v H over N columns, PER consecutive ones a lane: N / PER lanes a row
template <int N, int PER = 16, typename Acc>
__device__ __forceinline__ void fwht_lanes(Acc* v, int lane) {
#pragma unroll
  for (int h = 1; h < PER; h <<= 1)
#pragma unroll
    for (int r = 0; r < PER; ++r) {
      if (r & h) continue;
      const Acc a = v[r], c = v[r + h];
      v[r] = a + c;
      v[r + h] = a - c;
    }
  if constexpr (N / PER > 1) butterfly_lanes<1, PER>(v, lane);
  if constexpr (N / PER > 2) butterfly_lanes<2, PER>(v, lane);
  if constexpr (N / PER > 4) butterfly_lanes<4, PER>(v, lane);
  if constexpr (N / PER > 8) butterfly_lanes<8, PER>(v, lane);
}

// two fp32 as bf16, rounded to nearest even, in one instruction
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p = __builtin_convertvector((f32x2{lo, hi}), bf16x2);
  uint32_t w;
  __builtin_memcpy(&w, &p, 4);
  return w;
}

// 16 bytes or 16 values, consecutive, as fp32 or bf16 (rounded to nearest even);
// STREAM: past the caches, for outputs larger than they are
template <bool STREAM = false, typename TOut>
__device__ __forceinline__ void store_16b(TOut* dst, const float* f) {
  typedef float f32x4v __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
  if constexpr (sizeof(TOut) == 4) {
    f32x4v* p = reinterpret_cast<f32x4v*>(dst);
    const f32x4v x = f32x4v{f[0], f[1], f[2], f[3]};
    if constexpr (STREAM) __builtin_nontemporal_store(x, p); else *p = x;
  } else {
    u32x4v* p = reinterpret_cast<u32x4v*>(dst);
    const u32x4v x = u32x4v{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                            pack_bf16(f[6], f[7])};
    if constexpr (STREAM) __builtin_nontemporal_store(x, p); else *p = x;
  }
}
template <typename TOut>
__device__ __forceinline__ void store16(TOut* dst, const float* f) {
  constexpr int COLS = 16 / sizeof(TOut);
#pragma unroll
  for (int i = 0; i < 16 / COLS; ++i) store_16b(dst + i * COLS, f + i * COLS);
}

}  // namespace qwha
