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
// and read back as x' = s (q - z) H. A row that is not finite gets s = NaN and
// z = q = 0, so that whatever uses it shows it.
#include "cache.h"
#include "lane_fwht.h"

namespace qwha {

namespace {

// over the LANES lanes of a row
template <int LANES, bool MAX>
__device__ __forceinline__ float row_extreme(float m) {
  auto pick = [](float a, float b) { return MAX ? fmaxf(a, b) : fminf(a, b); };
  if constexpr (LANES > 1) m = pick(m, lane_xor<1>(m));
  if constexpr (LANES > 2) m = pick(m, lane_xor<2>(m));
  if constexpr (LANES > 4) m = pick(m, lane_xor<4>(m));
  if constexpr (LANES > 8) m = pick(m, lane_xor<8>(m));
  return m;
}

template <int LANES>
__device__ __forceinline__ float row_sum(float m) {
  if constexpr (LANES > 1) m += lane_xor<1>(m);
  if constexpr (LANES > 2) m += lane_xor<2>(m);
  if constexpr (LANES > 4) m += lane_xor<4>(m);
  if constexpr (LANES > 8) m += lane_xor<8>(m);
  return m;
}

// floor(v / s + 1/2) + add exactly, for |v| up to about 2^8 s. The quotient
// from the reciprocal is off by less than 2^-14, so q = floor(v/s + 1/2 - 2^-12)
// is the result or, beside a border, one below it; the residual r = v - q s, in
// [-s/2, s], then decides. One fma gives it: where |v| >= s both v and q s are
// multiples of ulp(s) and r is at most s, so it is exact; below, q is -1, 0 or 1
// and r is v, or v less or plus s, exact within a factor of two of each other and
// else on the side of s/2 that the exact difference is on, which rounding does
// not leave. The residual is doubled (exact) and not the step halved: half a step
// below 2^-125 may need a bit below fp32's smallest number. So the code is what
// infinite precision gives for this v and s, whatever computes it.
__device__ __forceinline__ int round_half_up(float v, float s, float inv, int add) {
  const float q = floorf(fmaf(v, inv, 0.5f - 0x1p-12f));
  const float r = fmaf(-q, s, v);
  return static_cast<int>(q) + add + (r + r >= s ? 1 : 0);
}

// Row `row` of a call's [T][2][heads] rows: keys, then values, head by head.
struct CallRow {
  uint32_t t;
  int part, head;
};
__device__ __forceinline__ CallRow call_row(const Cache& c, uint32_t row) {
  const uint32_t tp = c.over_heads(row);
  return CallRow{tp >> 1, static_cast<int>(tp & 1u), static_cast<int>(row - tp * c.heads)};
}

// Bound by the vector units and then HBM: a row reads N elements and writes
// N * b / 8 + 8 bytes. The transform runs in fp64: the sums of a row whose values
// lie within 2^37 (bf16) or 2^21 (fp32) of each other are then exact, so that v,
// its range and every code do not depend on the order of the additions. 32 columns
// a lane: a stage across lanes costs 3 to 5 instructions a value (two moves, a
// product and sum), one within a lane a single one. 8192 tokens of 8 heads of 128
// (33.5 MB of bf16 in, 9.4 out): 16.9 us (median of twelve), of which the vector
// units issue 31 instructions a value for 13.4 (at 2.4 GHz); at 4.9 TB/s the bytes
// take 8.8. As fp32 19.3 us, the bytes 15.6. 32 tokens: 4.1 us.
template <int N, int BITS, typename TIn, bool ROT>
__global__ __launch_bounds__(256) void cache_write_kernel(const TIn* __restrict__ k,
                                                          const TIn* __restrict__ v, uint32_t rows,
                                                          const int32_t* __restrict__ slots,
                                                          Cache c) {
  constexpr int PER = kWritePer, LPR = N / PER;
  constexpr int WORDS = PER * BITS / 32;
  constexpr float QMAX = static_cast<float>((1 << BITS) - 1);
  const int u = threadIdx.x % LPR;
  const uint32_t row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const CallRow cr = call_row(c, min(row, rows - 1));
  const int32_t slot = slots[cr.t];

  float f[PER];
  {
    const TIn* src = (cr.part ? v : k) +
                     (static_cast<uint64_t>(cr.t) * c.heads + cr.head) * N + u * PER;
    if constexpr (ROT) {
      double a[PER];
#pragma unroll
      for (int i = 0; i < PER / 16; ++i) load16(src + 16 * i, a + 16 * i);
      fwht_lanes<N, PER>(a, u);
#pragma unroll
      for (int r = 0; r < PER; ++r) f[r] = static_cast<float>(a[r] * (1. / N));   // the sum may pass fp32's range
    } else {
#pragma unroll
      for (int i = 0; i < PER / 16; ++i) load16(src + 16 * i, f + 16 * i);
    }
  }
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    lo = fminf(lo, f[r]);
    hi = fmaxf(hi, f[r]);
  }
  // NaN, which the extremes pass over, where a value is not finite (0 * f). The
  // transform adds every value of the row to each of its results: any one tells.
  float bad = 0.f * f[0];
  if constexpr (!ROT) {
#pragma unroll
    for (int r = 1; r < PER; ++r) bad = fmaf(0.f, f[r], bad);
    bad = row_sum<LPR>(bad);
  }
  lo = row_extreme<LPR, false>(lo);
  hi = row_extreme<LPR, true>(hi);
  float s = (hi - lo) / QMAX;
  const bool lost = !(s + bad < INFINITY);     // not finite, or a range past fp32's
  // a step below fp32's normal range holds nothing
  const bool flat = lost || !(s >= 1.17549435e-38f);
  if (flat) s = lost ? __builtin_nanf("") : 0.f;
  const float inv = flat ? 0.f : 1.f / s;
  const int z = flat ? 0 : round_half_up(-lo, s, inv, 0);
  uint32_t w[WORDS];
#pragma unroll
  for (int i = 0; i < WORDS; ++i) w[i] = 0u;
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int q = min(max(round_half_up(f[r], s, inv, z), 0), (1 << BITS) - 1);
    w[r * BITS / 32] |= static_cast<uint32_t>(q) << (r * BITS % 32);
  }
  if (row >= rows || slot < 0 || (slot >> c.lg_page) >= c.n_pages) return;
  const int64_t at = c.row(cr.part, slot, cr.head);
  uint4* dst = reinterpret_cast<uint4*>(c.codes + at * (N * BITS / 32) + u * WORDS);
#pragma unroll
  for (int i = 0; i < WORDS / 4; ++i)
    dst[i] = flat ? uint4{0u, 0u, 0u, 0u}
                  : uint4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
  if (u == 0) {
    c.scales[at] = s;
    c.zeros[at] = static_cast<float>(z);
  }
}

// The transform of 16 codes a lane, two to a register of 16-bit integers:
// sums of up to 256 codes of 4 bits, or of 8 bits less 128, fit them (for 8
// bits and 256 columns: 128 of each sign give at most 128 * 127 + 128 * 128,
// the row of ones at least -256 * 128), so the transform is exact and takes
// half the instructions. z and the 128 come back in column 0, the only one in
// which a constant row's transform is not zero.
typedef short s16x2 __attribute__((ext_vector_type(2)));

template <int X>
__device__ __forceinline__ s16x2 lane_xor_s16(s16x2 v) {
  int x;
  __builtin_memcpy(&x, &v, 4);
  x = lane_xor_i32<X>(x);
  __builtin_memcpy(&v, &x, 4);
  return v;
}
template <int X>
__device__ __forceinline__ void codes_lanes(s16x2* p, int lane) {
  const short one = lane & X ? -1 : 1;
  const s16x2 sign = s16x2{one, one};
#pragma unroll
  for (int r = 0; r < 8; ++r) p[r] = p[r] * sign + lane_xor_s16<X>(p[r]);
}

// w: 16 codes (2 or 4 words) -> f[16] = their transform, less 128 times
// N in column 0 for 8 bits
template <int N, int BITS>
__device__ __forceinline__ void transform_codes(const uint32_t* w, int lane, float* f) {
  constexpr int HALF = 16 / BITS;            // codes k and k + HALF of a word share a register
  constexpr uint32_t MASK = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu;
  s16x2 p[8];
#pragma unroll
  for (int i = 0; i < 16 * BITS / 32; ++i)
#pragma unroll
    for (int k = 0; k < HALF; ++k) {
      const uint32_t x = (w[i] >> (BITS * k)) & MASK;
      __builtin_memcpy(&p[i * HALF + k], &x, 4);
      if (BITS == 8) p[i * HALF + k] -= s16x2{128, 128};
    }
  // register index bits (the codes' bits but the one of the halves), the
  // halves, the lanes
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (r & h) continue;
      const s16x2 a = p[r], b = p[r + h];
      p[r] = a + b;
      p[r + h] = a - b;
    }
#pragma unroll
  for (int r = 0; r < 8; ++r) p[r] = p[r].yy * s16x2{1, -1} + p[r].xx;
  if constexpr (N > 16) codes_lanes<1>(p, lane);
  if constexpr (N > 32) codes_lanes<2>(p, lane);
  if constexpr (N > 64) codes_lanes<4>(p, lane);
  if constexpr (N > 128) codes_lanes<8>(p, lane);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int i = r / HALF * 2 * HALF + r % HALF;
    f[i] = static_cast<float>(p[r].x);
    f[i + HALF] = static_cast<float>(p[r].y);
  }
}

// Rows [T][2][heads] of the slots, dense; a token without a slot reads as
// zeros. Bound by HBM's writes: N elements out for N * b / 8 + 8 bytes in.
// Lane u of a row holds 16 bytes of output from each of SEGS places, N / SEGS
// columns apart (the transform takes the index bits in any order), so that a
// store instruction covers whole lines.
// IT rows a lane, their loads in flight together. Calls of many rows take 4 and
// store past the caches, whose lines the codes then keep: 40000 tokens of 8
// heads of 128 (209 MB) 49.1 us with one row and plain stores, 46.6 with 4 rows,
// 34.8 with stores past the caches too. With 64 columns a store instruction has
// but half of each line, which must meet the other half in the cache (16384 tokens
// of 8 heads of 64 as fp32: 21.0 us past it, 15.1 through it).
template <int N, int BITS, typename TOut, bool ROT, int IT>
__global__ __launch_bounds__(256) void cache_read_kernel(Cache c,
                                                         const int32_t* __restrict__ slots,
                                                         uint32_t rows, TOut* __restrict__ k,
                                                         TOut* __restrict__ v) {
  constexpr int LPR = N / 16, RPB = 256 / LPR, WORDS = 16 * BITS / 32;
  constexpr int COLS = 16 / sizeof(TOut), SEGS = 16 / COLS;
  const int u = threadIdx.x % LPR;
  const uint32_t row0 = blockIdx.x * (RPB * IT) + threadIdx.x / LPR;
  uint32_t w[IT][WORDS];
  float s[IT], z[IT];
  CallRow cr[IT];
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    cr[j] = call_row(c, min(row0 + j * RPB, rows - 1));
    const int32_t slot = slots[cr[j].t];
    const bool stored = slot >= 0 && (slot >> c.lg_page) < c.n_pages;
    const int64_t at = c.row(cr[j].part, stored ? slot : 0, cr[j].head);
    using Seg = std::conditional_t<COLS * BITS == 16, uint16_t,
                                   std::conditional_t<COLS * BITS == 32, uint32_t, uint2>>;
    const Seg* src = reinterpret_cast<const Seg*>(c.codes + at * (N * BITS / 32)) + u;
    Seg seg[SEGS];
#pragma unroll
    for (int i = 0; i < SEGS; ++i) seg[i] = src[i * LPR];
    __builtin_memcpy(w[j], seg, sizeof(seg));
    // a token without a slot: 0 times whatever finite codes slot 0 holds
    const float sv = c.scales[at], zv = c.zeros[at];
    s[j] = stored ? sv : 0.f;
    z[j] = stored ? zv : 0.f;
  }
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    float f[16];
    if constexpr (ROT) {
      transform_codes<N, BITS>(w[j], u, f);
      if (u == 0) f[0] += static_cast<float>(N) * ((BITS == 8 ? 128.f : 0.f) - z[j]);
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        f[r] = static_cast<float>((w[j][r * BITS / 32] >> (r * BITS % 32)) & ((1u << BITS) - 1u)) - z[j];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) f[r] *= s[j];
    if (row0 + j * RPB < rows) {
      TOut* dst = (cr[j].part ? v : k) +
                  (static_cast<uint64_t>(cr[j].t) * c.heads + cr[j].head) * N + u * COLS;
#pragma unroll
      for (int i = 0; i < SEGS; ++i) store_16b<IT == 4 && LPR >= 8>(dst + i * (N / SEGS), f + i * COLS);
    }
  }
}

// Elements from which on rows go 4 a lane (8 heads of 128, bf16, us with one / 4 a
// lane: 1024 tokens 3.2 / 3.8, 2048 4.2 / 3.8, 4096 6.8 / 5.1).
constexpr uint64_t kManyElements = 1u << 22;

}  // namespace

hipError_t launch_cache_write(const void* k, const void* v, Dt dt, int64_t T,
                              const int32_t* slots, int rotate, const Cache& c, hipStream_t s) {
  const uint32_t rows = static_cast<uint32_t>(T * 2 * c.heads);
  return by_shape(c.dim, c.bits, [&](auto n, auto bits) {
    constexpr int N = decltype(n)::value, BITS = decltype(bits)::value;
    constexpr int RPB = 256 / (N / kWritePer);
    const dim3 grid((rows - 1) / RPB + 1);
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
  const uint32_t rows = static_cast<uint32_t>(T * 2 * c.heads);
  return by_shape(c.dim, c.bits, [&](auto n, auto bits) {
    constexpr int N = decltype(n)::value, BITS = decltype(bits)::value, RPB = 256 / (N / 16);
    auto go = [&](auto it, auto rot, auto* kk, auto* vv) {
      using T = std::remove_pointer_t<decltype(kk)>;
      constexpr int IT = decltype(it)::value;
      hipLaunchKernelGGL((cache_read_kernel<N, BITS, T, decltype(rot)::value, IT>),
                         dim3((rows - 1) / (RPB * IT) + 1), dim3(256), 0, s, c, slots, rows, kk, vv);
      return hipGetLastError();
    };
    auto by_rows = [&](auto rot, auto* kk, auto* vv) {
      return static_cast<uint64_t>(rows) * N >= kManyElements ? go(std::integral_constant<int, 4>{}, rot, kk, vv)
                              : go(std::integral_constant<int, 1>{}, rot, kk, vv);
    };
    auto by_type = [&](auto rot) {
      if (dt == Dt::F32) return by_rows(rot, static_cast<float*>(k), static_cast<float*>(v));
      return by_rows(rot, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
    };
    return rotate ? by_type(std::true_type{}) : by_type(std::false_type{});
  });
}

}  // namespace qwha
