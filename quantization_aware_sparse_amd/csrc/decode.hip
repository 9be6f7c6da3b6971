// The quantized layer for the few tokens of a decoding step (QWHA notes,
// papernotes.org, 损失函数 / 训练策略; gist.science summary §4):
//   y = x W_Q^T + alpha z F^T,  z = FWHT(x) / b,  T <= 64 tokens.
// The weights' codes are read once for all tokens.
#include "common.h"
#include "launch.h"

namespace qwha {

namespace {

constexpr int kTok = 4;   // tokens per wave

// One wave per output row and kTok tokens.
template <typename T>
__global__ __launch_bounds__(256) void decode_rows_kernel(
    const T* __restrict__ x, int tokens, int K, int N, QuantW qw, const float* __restrict__ z,
    const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ E,
    const float* __restrict__ c, float alpha, T* __restrict__ y) {
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t0 = blockIdx.y * kTok;
  if (n >= N) return;
  float acc[kTok];
#pragma unroll
  for (int i = 0; i < kTok; ++i) acc[i] = 0.f;
  for (int j = lane; j < K; j += 64) {
    const uint32_t wi = __umulhi(static_cast<uint32_t>(j), qw.cpw_magic);
    const int sh = (j - static_cast<int>(wi) * qw.cpw) * qw.bits;
    const uint32_t w = qw.codes[static_cast<int64_t>(n) * qw.wpr + wi];
    const float code = static_cast<float>((w >> sh) & ((1u << qw.bits) - 1u));
    const int64_t g = static_cast<int64_t>(n) * qw.gpr + (j >> qw.lg_group);
    const float wv = (code - qw.zeros[g]) * qw.scales[g];
#pragma unroll
    for (int i = 0; i < kTok; ++i)
      if (t0 + i < tokens) acc[i] += wv * Elem<T>::ld(x, static_cast<int64_t>(t0 + i) * K + j);
  }
  if (z != nullptr) {
    const int k1 = row_ptr[n + 1];
    for (int k = row_ptr[n] + lane; k < k1; k += 64) {
      const int j = E[2 * static_cast<int64_t>(k) + 1];
      const float v = alpha * c[k];
#pragma unroll
      for (int i = 0; i < kTok; ++i)
        if (t0 + i < tokens) acc[i] += v * z[static_cast<int64_t>(t0 + i) * K + j];
    }
  }
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    float a = acc[i];
    for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o);
    if (lane == 0 && t0 + i < tokens) Elem<T>::st(y, static_cast<int64_t>(t0 + i) * N + n, a);
  }
}

}  // namespace

hipError_t launch_decode(const void* x, Dt dt, int T, int K, int N, const QuantW& qw,
                         const float* z, const int32_t* row_ptr, const int32_t* E,
                         const float* c, float alpha, void* y, hipStream_t s) {
  const dim3 grid((N + 3) / 4, (T + kTok - 1) / kTok);
  if (dt == Dt::F32)
    hipLaunchKernelGGL((decode_rows_kernel<float>), grid, dim3(256), 0, s,
                       static_cast<const float*>(x), T, K, N, qw, z, row_ptr, E, c, alpha,
                       static_cast<float*>(y));
  else
    hipLaunchKernelGGL((decode_rows_kernel<uint16_t>), grid, dim3(256), 0, s,
                       static_cast<const uint16_t*>(x), T, K, N, qw, z, row_ptr, E, c, alpha,
                       static_cast<uint16_t*>(y));
  return hipGetLastError();
}

}  // namespace qwha
