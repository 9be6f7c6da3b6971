// The quantized key/value cache: rows written and read back (attention over
// them: cache_attn.hip).
//
// A row is the head_dim values of one token's key or value of one head. With
// the transform on, what is stored is v = fp32(x H / n), n = head_dim, H the
// Sylvester matrix (QWHA notes, papernotes.org, 关键设计 1): H spreads a
// channel that stands out over the whole row, so that one scale and zero per
// row suffice. v is quantized to b bits over its range with zero included:
//   lo = min(v, 0), hi = max(v, 0), s = fp32(fp32(hi - lo) / (2^b - 1)),
//   z = floor(-lo/s + 1/2), q = clip(floor(v/s + 1/2) + z, 0, 2^b - 1),
// and read back as x' = s (q - z) H.
#include "cache.h"
#include "lane_fwht.h"

namespace qwha {

namespace {

template <int N, bool MAX>
__device__ __forceinline__ float row_extreme(float m) {
  auto pick = [](float a, float b) { return MAX ? fmaxf(a, b) : fminf(a, b); };
  if constexpr (N > 16) m = pick(m, lane_xor<1>(m));
  if constexpr (N > 32) m = pick(m, lane_xor<2>(m));
  if constexpr (N > 64) m = pick(m, lane_xor<4>(m));
  if constexpr (N > 128) m = pick(m, lane_xor<8>(m));
  return m;
}

// floor(v / s + 1/2) exactly, for |v| up to about 2^8 s: rint(v * (1/s)) is
// at most one off, and the residual v - q s is exact in one fma. (Its bits:
// where |v| >= s both v and q s are multiples of ulp(s) and the difference is
// at most about s; below, q is 0 or +-1 and the difference is exact as one of
// two numbers within a factor of two of each other.) So the comparison with
// s / 2 decides the rounding as infinite precision would, and equal inputs
// give equal codes whatever computes them.
__device__ __forceinline__ float round_half_up(float v, float s, float inv) {
  float q = rintf(v * inv);
  const float r = fmaf(-q, s, v), h = 0.5f * s;
  if (r >= h) q += 1.f;
  if (r < -h) q -= 1.f;
  return q;
}

// Written per token: keys, then values, head by head (the order of x).
// Bound by HBM: a row reads head_dim elements and writes head_dim * b / 8 + 8
// bytes. The transform runs in fp64: a row's sums are then exact (16-bit
// inputs whose exponents span less than 2^37), so v, its range and every code
// do not depend on the order of the additions.
template <int N, int BITS, typename TIn, bool ROT>
__global__ __launch_bounds__(256) void cache_write_kernel(const TIn* __restrict__ k,
                                                          const TIn* __restrict__ v, int64_t rows,
                                                          const int32_t* __restrict__ slots,
                                                          Cache c) {
  constexpr int LPR = N / 16;                  // lanes per row
  constexpr float QMAX = static_cast<float>((1 << BITS) - 1);
  const int u = threadIdx.x % LPR;
  // rows: [T][2][heads]
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
  const bool live = row < rows;
  const int64_t rr = live ? row : rows - 1;
  const int64_t tp = rr / c.heads;
  const int h = static_cast<int>(rr - tp * c.heads);
  const int part = static_cast<int>(tp & 1);
  const int64_t t = tp >> 1;
  const int32_t slot = slots[t];
  const bool stored = live && slot >= 0 && (slot >> c.lg_page) < c.n_pages;

  float f[16];
  {
    const TIn* src = (part ? v : k) + (t * c.heads + h) * N + u * 16;
    if constexpr (ROT) {
      double a[16];
      load16(src, a);
      fwht_lanes<N>(a, u);
#pragma unroll
      for (int r = 0; r < 16; ++r) f[r] = static_cast<float>(a[r] * (1.0 / N));
    } else {
      load16(src, f);
    }
  }
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    lo = fminf(lo, f[r]);
    hi = fmaxf(hi, f[r]);
  }
  lo = row_extreme<N, false>(lo);
  hi = row_extreme<N, true>(hi);
  float s = (hi - lo) / QMAX;
  const bool flat = !(s >= 1.17549435e-38f);   // a step below fp32's normal range holds nothing
  if (flat) s = 0.f;
  const float inv = flat ? 0.f : 1.f / s;
  const float z = flat ? 0.f : round_half_up(-lo, s, inv);
  uint32_t w[16 * BITS / 32];
#pragma unroll
  for (int i = 0; i < 16 * BITS / 32; ++i) w[i] = 0u;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float q = flat ? 0.f : fminf(fmaxf(round_half_up(f[r], s, inv) + z, 0.f), QMAX);
    w[r * BITS / 32] |= static_cast<uint32_t>(q) << (r * BITS % 32);
  }
  if (!stored) return;
  const int64_t at = c.row(part, slot, h);
  uint32_t* dst = c.codes + at * (N * BITS / 32) + u * (16 * BITS / 32);
  if constexpr (BITS == 4) {
    *reinterpret_cast<uint2*>(dst) = uint2{w[0], w[1]};
  } else {
    *reinterpret_cast<uint4*>(dst) = uint4{w[0], w[1], w[2], w[3]};
  }
  if (u == 0) {
    c.scales[at] = s;
    c.zeros[at] = z;
  }
}

// Rows [T][2][heads] of the slots, dense; a token without a slot reads as
// zeros. Bound by HBM's writes: head_dim elements out for head_dim * b / 8 + 8
// bytes in.
template <int N, int BITS, typename TOut, bool ROT>
__global__ __launch_bounds__(256) void cache_read_kernel(Cache c,
                                                         const int32_t* __restrict__ slots,
                                                         int64_t rows, TOut* __restrict__ k,
                                                         TOut* __restrict__ v) {
  constexpr int LPR = N / 16;
  const int u = threadIdx.x % LPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
  const bool live = row < rows;
  const int64_t rr = live ? row : rows - 1;
  const int64_t tp = rr / c.heads;
  const int h = static_cast<int>(rr - tp * c.heads);
  const int part = static_cast<int>(tp & 1);
  const int64_t t = tp >> 1;
  const int32_t slot = slots[t];
  float f[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) f[r] = 0.f;
  if (slot >= 0 && (slot >> c.lg_page) < c.n_pages) {
    const int64_t at = c.row(part, slot, h);
    const uint32_t* src = c.codes + at * (N * BITS / 32) + u * (16 * BITS / 32);
    uint32_t w[16 * BITS / 32];
    if constexpr (BITS == 4) {
      const uint2 p = *reinterpret_cast<const uint2*>(src);
      w[0] = p.x; w[1] = p.y;
    } else {
      const uint4 p = *reinterpret_cast<const uint4*>(src);
      w[0] = p.x; w[1] = p.y; w[2] = p.z; w[3] = p.w;
    }
    const float s = c.scales[at], z = c.zeros[at];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint32_t q = (w[r * BITS / 32] >> (r * BITS % 32)) & ((1u << BITS) - 1u);
      f[r] = (static_cast<float>(q) - z) * s;
    }
  }
  // every lane of a row takes the same branch above, so the butterflies see whole rows
  if constexpr (ROT) fwht_lanes<N>(f, u);
  if (live) store16((part ? v : k) + (t * c.heads + h) * N + u * 16, f);
}

}  // namespace

hipError_t launch_cache_write(const void* k, const void* v, Dt dt, int64_t T,
                              const int32_t* slots, int rotate, const Cache& c, hipStream_t s) {
  const int64_t rows = T * 2 * c.heads;
  return by_shape(c.dim, c.bits, [&](auto n, auto bits) {
    constexpr int N = decltype(n)::value, BITS = decltype(bits)::value;
    const dim3 grid(static_cast<unsigned>((rows * (N / 16) + 255) / 256));
    auto go = [&](auto kernel, auto* kk, auto* vv) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, kk, vv, rows, slots, c);
      return hipGetLastError();
    };
    if (dt == Dt::F32) {
      auto* kk = static_cast<const float*>(k);
      auto* vv = static_cast<const float*>(v);
      return rotate ? go(cache_write_kernel<N, BITS, float, true>, kk, vv)
                    : go(cache_write_kernel<N, BITS, float, false>, kk, vv);
    }
    auto* kk = static_cast<const uint16_t*>(k);
    auto* vv = static_cast<const uint16_t*>(v);
    return rotate ? go(cache_write_kernel<N, BITS, uint16_t, true>, kk, vv)
                  : go(cache_write_kernel<N, BITS, uint16_t, false>, kk, vv);
  });
}

hipError_t launch_cache_read(const Cache& c, const int32_t* slots, int64_t T, int rotate, Dt dt,
                             void* k, void* v, hipStream_t s) {
  const int64_t rows = T * 2 * c.heads;
  return by_shape(c.dim, c.bits, [&](auto n, auto bits) {
    constexpr int N = decltype(n)::value, BITS = decltype(bits)::value;
    const dim3 grid(static_cast<unsigned>((rows * (N / 16) + 255) / 256));
    auto go = [&](auto kernel, auto* kk, auto* vv) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, c, slots, rows, kk, vv);
      return hipGetLastError();
    };
    if (dt == Dt::F32) {
      auto* kk = static_cast<float*>(k);
      auto* vv = static_cast<float*>(v);
      return rotate ? go(cache_read_kernel<N, BITS, float, true>, kk, vv)
                    : go(cache_read_kernel<N, BITS, float, false>, kk, vv);
    }
    auto* kk = static_cast<uint16_t*>(k);
    auto* vv = static_cast<uint16_t*>(v);
    return rotate ? go(cache_read_kernel<N, BITS, uint16_t, true>, kk, vv)
                  : go(cache_read_kernel<N, BITS, uint16_t, false>, kk, vv);
  });
}

}  // namespace qwha
