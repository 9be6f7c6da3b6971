// The Walsh-Hadamard transform of rows that lie across the lanes of a wave:
// out[j] = sum_m in[m] * (-1)^popcount(m & j), N = 64, 128 or 256 columns,
// 16 consecutive ones a lane, N / 16 neighbouring lanes a row.
#pragma once

#include "common.h"

namespace qwha {

template <int X, typename Acc>
__device__ __forceinline__ void butterfly_lanes(Acc* v, int lane) {
  const bool upper = (lane & X) != 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const Acc o = lane_xor<X>(v[r]);
    v[r] = upper ? o - v[r] : v[r] + o;
  }
}

// v H over N columns, 16 a lane
template <int N, typename Acc>
__device__ __forceinline__ void fwht_lanes(Acc* v, int lane) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (r & h) continue;
      const Acc a = v[r], c = v[r + h];
      v[r] = a + c;
      v[r + h] = a - c;
    }
  if constexpr (N > 16) butterfly_lanes<1>(v, lane);
  if constexpr (N > 32) butterfly_lanes<2>(v, lane);
  if constexpr (N > 64) butterfly_lanes<4>(v, lane);
  if constexpr (N > 128) butterfly_lanes<8>(v, lane);
}

// 16 consecutive values as fp32 or bf16 (rounded to nearest even)
template <typename TOut>
__device__ __forceinline__ void store16(TOut* dst, const float* f) {
  if constexpr (sizeof(TOut) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = float4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(f[2 * i])) |
             (static_cast<uint32_t>(f32_to_bf16(f[2 * i + 1])) << 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<uint4*>(dst)[i] = uint4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
  }
}

}  // namespace qwha
