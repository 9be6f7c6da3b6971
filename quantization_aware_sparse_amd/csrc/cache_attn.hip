// Attention of one query token per sequence over the quantized cache:
//   out = sum_t softmax_t(scale q . k_t) v_t,  k_t = s (code - z) H (H = 1
// without the transform). H is symmetric, so q . k_t = (q H) . (s (code - z)):
// the query is transformed once instead of every key, and the sum over the
// values' codes once instead of every value.
//
// A workgroup takes one key/value head of one sequence, up to 4 HT of the query
// heads that read it, and a slice of the tokens; its waves take tiles of 32
// tokens in turn, each with its own running maximum and sum of the softmax.
//   scores  on the 8-bit integer matrix cores (v_mfma_i32_16x16x64_i8), exact.
//           A: 16 rows = 4 query heads x 4 signed digits of 8 bits: q' is rounded
//           to a whole number of 2^(e - 31), 2^e the power of two above the head's
//           largest |q'|. That keeps all 24 bits of components of 2^-6 of the
//           largest and more, and leaves the others an error of 1.02 * 2^-31 of it
//           at most, 1/128 of what one rounding of an fp32 sum with the largest in
//           it costs. B: 16 tokens' codes (8-bit ones less 128). Codes need a mask
//           and a shift to be operands, as bf16 a permutation and an or of each
//           pair as well. Lane l holds token l % 16 and a quarter of its row;
//   values  on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16). A: the weights
//           p s_v as three bf16 numbers that sum to them exactly; B: for each of
//           N / 16 columns j the codes of column (N / 16) (l % 16) + j of 8
//           tokens: a lane reads its N / 16 columns of 8 tokens and pairs the
//           tokens' codes up, as 16 + q (4 bits) or q (8 bits), exact in bf16.
// What is constant in (q - z) is taken off in fp32:
//   score   = s_k sum_i 256^(3-i) (sum d_i code' + (0 or 128 - z_k) sum d_i), digit
//             sums d_i by digit sums: whole numbers below 2^24 for whole z_k, so a
//             column whose code is its zero point leaves nothing, however large q';
//   output  = sum p s_v (OFF + code) - sum p s_v (OFF + z_v).
// A head's parts lie in one lane's results.
// Bound by the bytes, and by the waves' waits for them between the vector
// instructions that unpack: about 290 of a wave for 32 tokens of 128 columns, 9 KB
// of 4-bit keys and values. Measured (median device time of twelve runs; the cache's
// bytes at the 4.9 TB/s of a copy): 32 sequences of 1900 .. 4096 tokens, 8 x 4 heads
// of 128, 4 bits 31.5 us of 22.7, of which vector instructions issue for 13.8 (at 2.4
// GHz) and the matrix cores are busy for 1.9; waves wait half of their cycles. 3 of up
// to 30001, 16 x 1 heads of 64, 8 bits 26.8 + 4.8 us of 21, 9.2 of them issue; one of
// 777, 8 x 4 heads of 128 5.7 + 4.0 us of 0.2.
//
// cache_combine_kernel joins the slices: one maximum, one sum, one transform.
//
// A row without tokens is known by a sum of exactly 0. What is not finite is
// passed on: a NaN score is in the sums though not in the maximum, +inf makes
// its own weight NaN; -inf, from finite rows whose product passes fp32's range,
// weighs nothing.
#include <algorithm>

#include "cache.h"
#include "lane_fwht.h"
#include "mfma_codes.h"

namespace qwha {

namespace {

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * 64;
// waves of a workgroup that takes a short sequence alone; 16 need 128 registers
constexpr int many_waves(int n, int bits, int ht) { return ht == 1 && n * bits <= 512 ? 16 : 8; }
constexpr int kMaxWaves = 16;
constexpr int kTile = 32;                           // tokens
constexpr int kTabPages = 1024;                     // pages a slice holds, at most
constexpr int kTab = kTabPages + kMaxWaves * kTile / 8 + 1;

struct AttnArgs {
  int q_heads, per, groups;    // query heads per key/value head, in groups of 4 HT
  const int32_t* table;
  int width;
  const int32_t* lens;
  float scale;                 // times log2 e: the softmax runs on powers of two
  int rotate, slices;
  float* part;                 // [B][q_heads][slices][N]
  float2* ml;                  // [B][q_heads][slices]: maximum, sum
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// over the 16 lanes of a quarter
__device__ __forceinline__ float quarter_max(float v) {
  v = fmaxf(v, lane_xor<1>(v));
  v = fmaxf(v, lane_xor<2>(v));
  v = fmaxf(v, lane_xor<4>(v));
  return fmaxf(v, lane_xor<8>(v));
}
__device__ __forceinline__ uint32_t quarter_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(lane_xor_i32<1>(static_cast<int>(v))));
  v = max(v, static_cast<uint32_t>(lane_xor_i32<2>(static_cast<int>(v))));
  v = max(v, static_cast<uint32_t>(lane_xor_i32<4>(static_cast<int>(v))));
  return max(v, static_cast<uint32_t>(lane_xor_i32<8>(static_cast<int>(v))));
}
__device__ __forceinline__ float quarter_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  return v + lane_xor<8>(v);
}

// A lane's part of fp32 numbers: what is left after taking off the upper 8 bits
// of mantissa (`first` lanes: 0xFFFF0000) and the next 8 (`second` lanes), cut to
// bf16. Without branches; rows of no part hold a copy that nobody reads.
struct PartMask {
  uint32_t first, second;
  __device__ __forceinline__ explicit PartMask(int part)
      : first(part >= 1 ? 0xFFFF0000u : 0u), second(part >= 2 ? 0xFFFF0000u : 0u) {}
};
__device__ __forceinline__ bf16x8 part_operand(const float* f, PartMask m) {
  uint32_t x[8], d[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = f[i] - __uint_as_float(__float_as_uint(f[i]) & m.first);
    x[i] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & m.second));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
  return as_operand(d);
}

template <int WORDS>
__device__ __forceinline__ void load_words(const char* p, uint32_t* w) {
  if constexpr (WORDS >= 4) {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// o[N] in LDS -> out, through the transform: N / 16 lanes
template <int N, typename T>
__device__ __forceinline__ void finish_row(const float* o, int u, int rotate, T* out) {
  float v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = o[u * 16 + r];
  if (rotate) fwht_lanes<N>(v, u);
  store16(out + u * 16, v);
}

// ONE_PAGE: a tile lies in one page (of 32 tokens or more), whose address the
// whole wave shares.
template <int N, int BITS, int HT, bool ONE_PAGE, int WAVES, typename T>
__global__ __launch_bounds__(WAVES * 64, 2) void cache_attn_kernel(const T* __restrict__ q,
                                                                     Cache c, AttnArgs a,
                                                                     T* __restrict__ out) {
  constexpr int HEADS = 4 * HT, THREADS = WAVES * 64;
  constexpr int STEPS = N / 64;                     // matrix instructions of a score
  constexpr int KW = N / 4 * BITS / 32;             // words of a quarter of a row
  constexpr int J = N / 16;                         // columns of a lane
  constexpr int VB = J * BITS / 8;                  // bytes of them
  constexpr int VW = VB >= 4 ? VB / 4 : 1;
  constexpr int ROW = N * BITS / 8;                 // bytes of a row
  constexpr float OFF = BITS == 4 ? 16.f : 0.f;     // in the values' operands
  constexpr float KOFF = BITS == 4 ? 0.f : 128.f;   // taken off the keys'

  constexpr int PLD = kTile + 4;
  __shared__ __attribute__((aligned(16))) float qs[HEADS][N];
  __shared__ __attribute__((aligned(16))) float om[WAVES][HEADS][N];
  __shared__ float2 wml[WAVES][HEADS];
  __shared__ int32_t tab[kTab];
  float (*ps)[4][PLD] = reinterpret_cast<float (*)[4][PLD]>(&om[threadIdx.x >> 6][0][0]);
  static_assert(HT * 4 * PLD <= HEADS * N, "a wave's weights fit its place for results");

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int b = blockIdx.y;
  const int slice = blockIdx.x % a.slices, hg = blockIdx.x / a.slices;
  const int h = hg / a.groups, h0 = hg % a.groups * HEADS;     // key/value head, first query head
  const int heads = min(HEADS, a.per - h0);
  const int64_t qrow = static_cast<int64_t>(b) * a.q_heads + static_cast<int64_t>(h) * a.per + h0;

  const int64_t cap = static_cast<int64_t>(a.width) << c.lg_page;
  const int64_t asked = a.lens[b];
  const uint32_t len = static_cast<uint32_t>(asked < 0 ? 0 : asked < cap ? asked : cap);
  const uint32_t tiles = (len + kTile - 1) / kTile;
  uint32_t each = (tiles + a.slices - 1) / a.slices;
  each = (each + WAVES - 1) & ~(WAVES - 1u);
  const uint32_t first = min(static_cast<uint64_t>(slice) * each, static_cast<uint64_t>(tiles));
  const uint32_t last = min(first + each, tiles);

  // the slice's pages; one outside the cache, and those behind the sequence, as -1
  const uint32_t p0 = (first * kTile) >> c.lg_page;
  {
    const uint32_t pages = (len + (1u << c.lg_page) - 1) >> c.lg_page;
    const uint32_t p1 = (last * kTile + (1u << c.lg_page) - 1) >> c.lg_page;
    const int32_t* row = a.table + static_cast<int64_t>(b) * a.width;
    for (uint32_t p = p0 + tid; p < p1; p += THREADS) {
      const int32_t g = p < pages ? row[p] : -1;
      tab[p - p0] = g >= 0 && g < c.n_pages ? g : -1;
    }
  }
  if (tid < HEADS * J) {                            // one wave, N / 16 lanes a head
    const int head = tid / J, u = tid % J;
    float v[16];
    load16(q + (qrow + min(head, heads - 1)) * N + u * 16, v);
    if (a.rotate) fwht_lanes<N>(v, u);
#pragma unroll
    for (int r = 0; r < 16; ++r) qs[head][u * 16 + r] = v[r] * a.scale;
  }
  __syncthreads();

  const PartMask pm(lr & 3);
  const uint32_t pick = 0x0703u - 0x0101u * (lr & 3);   // the lane's digit of two numbers
  // digits of the queries: q' = 2^(e - 31) Q with 0.99 * 2^e above the head's
  // largest |q'|, so that Q = ((d0 256 + d1) 256 + d2) 256 + d3 in digits of
  // -128 .. 127.
  // Lane l: row l % 16 = (head, digit), the columns of its quarter in the order
  // of the codes' operands.
  i32x4 qf[HT][STEPS];
  int qexp[HT];                                     // of head lq: e - 31,
  float dsum[HT][3];                                // sums of d0, d1 and d2 256 + d3
  const i32x4 izero4 = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < HT; ++t) {
    // as bits, in which infinities and NaN are above all numbers
    auto largest = [&](int head) {
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < J; ++i) top = max(top, __float_as_uint(fabsf(qs[head][lr * J + i])));
      return quarter_max(top);
    };
    // the maximum of head t * 4 + lq is at hand in quarter lq, that of the
    // lane's row, head lr / 4, in quarter lr / 4
    const uint32_t top = largest(t * 4 + lq);
    const int finite = top < 0x7F800000u;
    const float largest_q = finite ? __uint_as_float(top) : 0.f;
    const int e = __builtin_amdgcn_frexp_expf(largest_q) +
                  (__builtin_amdgcn_frexp_mantf(largest_q) > 0.99f ? 1 : 0);
    qexp[t] = e - 31;
    const int up = 31 - __shfl(e, (lr >> 2) * 16), whole = __shfl(finite, (lr >> 2) * 16);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // column of byte i of register r: 4-bit words give their even codes
          // first, then their odd ones
          const int at = BITS == 4 ? r / 2 * 8 + 2 * i + r % 2 : r * 4 + i;
          const float f = rintf(__builtin_amdgcn_ldexpf(
              qs[t * 4 + (lr >> 2)][lq * (N / 4) + s * 16 + at], up));
          // Q + 128 (256^3 + 256^2 + 256 + 1) has the digits, each with 128 added
          b[i] = static_cast<uint32_t>(whole ? static_cast<int>(f) : 0) + 0x80808080u;
        }
        const uint32_t x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], pick),
                                                 __builtin_amdgcn_perm(b[1], b[0], pick),
                                                 0x05040100u) ^ 0x80808080u;
        qf[t][s][r] = static_cast<int>(x);
      }
    const i32x4 iones4 = i32x4{0x01010101, 0x01010101, 0x01010101, 0x01010101};
    i32x4 ds = izero4;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      ds = __builtin_amdgcn_mfma_i32_16x16x64_i8(qf[t][s], iones4, ds, 0, 0, 0);
    dsum[t][0] = static_cast<float>(ds[0]);
    dsum[t][1] = static_cast<float>(ds[1]);
    // NaN makes every score of the head NaN
    dsum[t][2] = finite ? static_cast<float>(ds[2] * 256 + ds[3]) : __builtin_nanf("");
  }

  const uint32_t mask = in_vgpr(kMask4);
  const f32x4 zero4 = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t vals = c.part_rows();
  const uint32_t in_page = (1u << c.lg_page) - 1;
  f32x4 acc[HT][J];
  float m[HT], l[HT];
#pragma unroll
  for (int t = 0; t < HT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) acc[t][j] = zero4;
  }

  struct Tile {
    uint32_t k[2][KW], v[8][VW];
    float sk[2], zk[2], sv[2], zv[2];
    bool live[2];
  };
  auto row_of = [&](uint32_t t, bool* live) {       // clamped to the cache's first page
    const int32_t g = tab[(t >> c.lg_page) - p0];
    *live = t < len && g >= 0;
    return c.row_in(0, g < 0 ? 0 : g, static_cast<int>(t & in_page), h);
  };
  const uint32_t koff = lr * ROW + lq * (ROW / 4), voff = 8 * lq * ROW + lr * VB;
  auto fetch_page = [&](Tile& x, uint32_t tile) {
    const uint32_t t = tile * kTile;
    const int32_t g = __builtin_amdgcn_readfirstlane(tab[(t >> c.lg_page) - p0]);
    const int64_t r = c.row_in(0, g < 0 ? 0 : g, static_cast<int>(t & in_page), h);
    const char* kp = reinterpret_cast<const char*>(c.codes) + r * ROW;
    const char* vp = kp + vals * ROW;
    const float *sp = c.scales + r, *zp = c.zeros + r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x.live[i] = g >= 0 && t + 16 * i + lr < len;
      load_words<KW>(kp + (koff + 16 * i * ROW), x.k[i]);
      x.sk[i] = sp[16 * i + lr];
      x.zk[i] = zp[16 * i + lr];
      x.sv[i] = (sp + vals)[16 * i + lr];
      x.zv[i] = (zp + vals)[16 * i + lr];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (VB >= 4)
        load_words<VW>(vp + (voff + i * ROW), x.v[i]);
      else
        x.v[i][0] = *reinterpret_cast<const uint16_t*>(vp + (voff + i * ROW));
    }
  };
  auto fetch = [&](Tile& x, uint32_t tile) {
    if constexpr (ONE_PAGE) {
      fetch_page(x, tile);
      return;
    }
    const char* codes = reinterpret_cast<const char*>(c.codes);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = row_of(tile * kTile + 16 * i + lr, &x.live[i]);
      load_words<KW>(codes + r * ROW + lq * (ROW / 4), x.k[i]);
      x.sk[i] = c.scales[r];
      x.zk[i] = c.zeros[r];
      x.sv[i] = c.scales[vals + r];
      x.zv[i] = c.zeros[vals + r];
    }
    // 8 tokens of one page (8 divides the page)
    bool any;
    const char* vp = codes + (vals + row_of(tile * kTile + 8 * lq, &any)) * ROW + lr * VB;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (VB >= 4)
        load_words<VW>(vp + i * ROW, x.v[i]);
      else
        x.v[i][0] = *reinterpret_cast<const uint16_t*>(vp + i * ROW);
    }
  };

  Tile cur;
  if (first + w < last) fetch(cur, first + w);
#pragma unroll 1
  for (uint32_t tile = first + w; tile < last; tile += WAVES) {
    Tile next;
    if (tile + WAVES < last) fetch(next, tile + WAVES);

    i32x4 sg[HT][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        i32x4 kf;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (BITS == 4) {
            const uint32_t w = cur.k[i][2 * s + r / 2];
            kf[r] = static_cast<int>((r % 2 ? w >> 4 : w) & 0x0F0F0F0Fu);
          } else {
            kf[r] = static_cast<int>(cur.k[i][4 * s + r] ^ 0x80808080u);
          }
        }
#pragma unroll
        for (int t = 0; t < HT; ++t)
          sg[t][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(qf[t][s], kf, s ? sg[t][i] : izero4, 0, 0, 0);
      }
    // what lies in a place that is left out is never used, whatever it holds
    float sv[2], ov[2], lost[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // 0, or NaN where a key's step or zero is not finite: its score is then NaN,
      // and not an infinity that might weigh nothing
      lost[i] = fmaf(0.f, cur.sk[i], 0.f * cur.zk[i]);
      sv[i] = cur.live[i] ? cur.sv[i] : 0.f;
      ov[i] = cur.live[i] ? OFF + cur.zv[i] : 0.f;
    }
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      float s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // the lower two digits together, below 2^31: their rounding to fp32 is less
        // than what rounding q' to whole numbers costs
        const float z = KOFF - cur.zk[i];
        const float d0 = fmaf(z, dsum[t][0], static_cast<float>(sg[t][i][0]));
        const float d1 = fmaf(z, dsum[t][1], static_cast<float>(sg[t][i][1]));
        const float d2 = fmaf(z, dsum[t][2], static_cast<float>(sg[t][i][2] * 256 + sg[t][i][3]));
        // the step takes the power of two: where that passes below fp32's range the
        // score is 0 to within 2^-100
        const float x = fmaf(__builtin_amdgcn_ldexpf(cur.sk[i], qexp[t]),
                             fmaf(0x1p24f, d0, fmaf(0x1p16f, d1, d2)), lost[i]);
        s[i] = cur.live[i] ? x : -INFINITY;
      }
      const float mn = fmaxf(m[t], quarter_max(fmaxf(s[0], s[1])));
      const float at = mn == -INFINITY ? 0.f : mn;    // nothing to see yet: all weights are 0
      if (__any(mn > m[t])) {
        const float keep = exp2_fast(m[t] - at);
        l[t] *= keep;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][j][r] *= keep;
        m[t] = mn;
      }
      float zs = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float p = exp2_fast(s[i] - at);
        l[t] += p;
        const float pv = p * sv[i];
        zs = fmaf(pv, ov[i], zs);
        ps[t][lq][16 * i + lr] = pv;
      }
      // sum p s_v (OFF + z_v) comes off tile by tile, ahead of the tile's product:
      // what adds up over the tokens is then the output itself, and not the far
      // larger sums that it is the difference of
      zs = quarter_sum(zs);
#pragma unroll
      for (int j = 0; j < J; ++j) acc[t][j][0] -= zs;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bf16x8 pf[HT];
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      const float4* p = reinterpret_cast<const float4*>(&ps[t][lr >> 2][8 * lq]);
      const float4 p0v = p[0], p1v = p[1];
      const float f[8] = {p0v.x, p0v.y, p0v.z, p0v.w, p1v.x, p1v.y, p1v.z, p1v.w};
      pf[t] = part_operand(f, pm);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t d[4];
      if constexpr (BITS == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = cur.v[2 * k][j / 8], hi = cur.v[2 * k + 1][j / 8];
          const uint32_t sel = 0x0C040C00u + 0x00010001u * (j % 8 / 2);
          d[k] = j % 2 ? and_or(__builtin_amdgcn_perm(hi >> 1, lo >> 1, sel), mask, kBase4)
                       : and_or(__builtin_amdgcn_perm(hi << 3, lo << 3, sel), mask, kBase4);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[k] = __builtin_amdgcn_perm(byte_f32(cur.v[2 * k + 1][j / 4], j % 4),
                                       byte_f32(cur.v[2 * k][j / 4], j % 4), 0x07060302u);
      }
      const bf16x8 vf = as_operand(d);
#pragma unroll
      for (int t = 0; t < HT; ++t)
        acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[t], vf, acc[t][j], 0, 0, 0);
    }
    cur = next;
  }

  // the waves' sums, joined
#pragma unroll
  for (int t = 0; t < HT; ++t) {
    const float ls = quarter_sum(l[t]);
#pragma unroll
    for (int j = 0; j < J; ++j)
      om[w][t * 4 + lq][lr * J + j] = acc[t][j][0] + acc[t][j][1] + acc[t][j][2];
    if (lr == 0) wml[w][t * 4 + lq] = float2{m[t], ls};
  }
  __syncthreads();
  for (int e = tid; e < heads * N; e += THREADS) {
    const int head = e / N, d = e % N;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, wml[i][head].x);
    // a NaN score is passed over by the maximum and stays in the sums
    const float at = top == -INFINITY ? 0.f : top;
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const float f = exp2_fast(wml[i][head].x - at);
      o = fmaf(f, om[i][head][d], o);
      sum = fmaf(f, wml[i][head].y, sum);
    }
    if (a.slices == 1) {
      qs[head][d] = sum == 0.f ? 0.f : o / sum;     // no tokens
    } else {
      const int64_t row = (qrow + head) * a.slices + slice;
      a.part[row * N + d] = o;
      if (d == 0) a.ml[row] = float2{top, sum};
    }
  }
  if (a.slices == 1) {
    __syncthreads();
    if (tid < heads * J) finish_row<N>(qs[tid / J], tid % J, a.rotate, out + (qrow + tid / J) * N);
  }
}

// One query head of one sequence: its slices, joined. N / 16 lanes read a slice's
// sums beside its maximum and sum; the workgroup's 16 * 256 / N such groups take
// the slices in turn, each with its own running maximum: one way to memory, and
// the groups meet in LDS.
template <int N, typename T>
__global__ __launch_bounds__(kAttnThreads) void cache_combine_kernel(AttnArgs a,
                                                                     T* __restrict__ out) {
  constexpr int J = N / 16, GROUPS = kAttnThreads / J;
  __shared__ float os[GROUPS][N + 4];
  __shared__ float2 gml[GROUPS];
  const int64_t row = static_cast<int64_t>(blockIdx.y) * a.q_heads + blockIdx.x;
  const int tid = threadIdx.x, u = tid % J, g = tid / J;
  float v[16], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = 0.f;
  for (int s = g; s < a.slices; s += GROUPS) {
    const float2 x = a.ml[row * a.slices + s];
    const float4* p = reinterpret_cast<const float4*>(a.part + (row * a.slices + s) * N + u * 16);
    float4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = p[i];
    if (x.y == 0.f) continue;                      // a slice without tokens; NaN goes on
    const float mn = fmaxf(top, x.x), keep = exp2_fast(top - mn), f = exp2_fast(x.x - mn);
    top = mn;
    sum = fmaf(f, x.y, sum * keep);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * i] = fmaf(f, o[i].x, v[4 * i] * keep);
      v[4 * i + 1] = fmaf(f, o[i].y, v[4 * i + 1] * keep);
      v[4 * i + 2] = fmaf(f, o[i].z, v[4 * i + 2] * keep);
      v[4 * i + 3] = fmaf(f, o[i].w, v[4 * i + 3] * keep);
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) os[g][u * 16 + r] = v[r];
  if (u == 0) gml[g] = float2{top, sum};
  __syncthreads();
  const int used = min(GROUPS, a.slices);
  if (tid < N) {
    top = -INFINITY;
    for (int i = 0; i < used; ++i) top = fmaxf(top, gml[i].x);
    const float at = top == -INFINITY ? 0.f : top;
    float o = 0.f, l = 0.f;
    for (int i = 0; i < used; ++i) {
      const float f = exp2_fast(gml[i].x - at);
      o = fmaf(f, os[i][tid], o);
      l = fmaf(f, gml[i].y, l);
    }
    os[0][tid] = l == 0.f ? 0.f : o / l;           // column tid is this thread's alone
  }
  __syncthreads();
  if (tid < J) finish_row<N>(os[0], u, a.rotate, out + row * N);
}

// Query heads of a workgroup: tiles of 4, two of them where there are more than
// 4 and the columns leave the registers for it.
int head_tiles(int per, int dim) { return per > 4 && dim <= 128 ? 2 : 1; }

// How the tokens are shared out. `many`: one workgroup of many waves for a
// sequence and key/value head, no joining pass. Else slices of a sequence:
// workgroups of 4 waves for four per compute unit, each with a tile for every
// wave, and no more pages than its table holds.
// The joining pass costs 3.5 us and up, while a compute unit alone takes 2 us a
// round of 512 tokens; the more workgroups there are, the less of the chip the
// first way leaves idle. Columns 128, 4 bits, 8 x 4 heads, us with one workgroup /
// with slices:
//   sequences   tokens  200         1000        2000        4000        8000
//    1           7.0 / 8.4  11.6 /  8.5  16.0 /  8.8  24.0 /  9.5  39.6 / 12.4
//   16                   -  12.9 / 15.5  18.1 / 17.9  27.0 / 22.9  46.2 / 39.6
//   32          7.5 / 11.8  14.3 / 18.8  20.4 / 23.8  36.9 / 40.8  64.9 / 69.3
// (32 of ragged lengths up to 8000: 50.0 / 48.0, up to 4000: 27.8 / 28.3).
struct AttnPlan {
  bool many;
  int slices;
};

AttnPlan attn_plan(int B, int q_heads, int heads, int dim, int64_t max_tokens, int page) {
  const int per = q_heads / heads, ht = head_tiles(per, dim);
  const int64_t groups = (per + 4 * ht - 1) / (4 * ht);
  const int64_t pairs = static_cast<int64_t>(B) * heads * groups;
  const int64_t one = kAttnWaves * kTile;           // tokens of a round of one workgroup
  if (max_tokens > one && pairs <= 256 && max_tokens <= std::max<int64_t>(256, pairs * pairs / 16))
    return {true, 1};
  const int64_t most = (max_tokens + one - 1) / one;
  const int64_t least = (max_tokens + kTabPages * static_cast<int64_t>(page) - 1) /
                        (kTabPages * static_cast<int64_t>(page));
  int64_t want = pairs > 0 ? (1024 + pairs - 1) / pairs : 1;
  if (want > most) want = most;
  if (want < least) want = least;
  return {false, static_cast<int>(want < 1 ? 1 : want)};
}

}  // namespace

size_t cache_attn_scratch_bytes(int B, int q_heads, int heads, int dim, int64_t max_tokens,
                                int page) {
  const int slices = attn_plan(B, q_heads, heads, dim, max_tokens, page).slices;
  if (slices == 1) return 0;
  return static_cast<size_t>(B) * q_heads * slices * (dim + 2) * sizeof(float);
}

int64_t cache_attn_blocks(int B, int q_heads, int heads, int dim, int64_t max_tokens, int page) {
  const int per = q_heads / heads, ht = head_tiles(per, dim);
  return static_cast<int64_t>(heads) * ((per + 4 * ht - 1) / (4 * ht)) *
         attn_plan(B, q_heads, heads, dim, max_tokens, page).slices;
}

hipError_t launch_cache_attn(const void* q, Dt dt, int B, int q_heads, const Cache& c,
                             const int32_t* table, int width, const int32_t* lens, float scale,
                             int rotate, void* out, void* scratch, hipStream_t s) {
  AttnArgs a;
  a.q_heads = q_heads;
  a.per = q_heads / c.heads;
  const int ht = head_tiles(a.per, c.dim);
  a.groups = (a.per + 4 * ht - 1) / (4 * ht);
  a.table = table;
  a.width = width;
  a.lens = lens;
  a.scale = scale * kLog2E;
  a.rotate = rotate;
  const AttnPlan plan = attn_plan(B, q_heads, c.heads, c.dim,
                                  static_cast<int64_t>(width) << c.lg_page, 1 << c.lg_page);
  a.slices = plan.slices;
  a.part = static_cast<float*>(scratch);
  a.ml = reinterpret_cast<float2*>(a.part + static_cast<int64_t>(B) * q_heads * a.slices * c.dim);
  const dim3 grid(static_cast<unsigned>(c.heads) * a.groups * a.slices, static_cast<unsigned>(B));
  return by_shape(c.dim, c.bits, [&](auto n, auto bits) {
    constexpr int N = decltype(n)::value, BITS = decltype(bits)::value;
    auto go = [&](auto* qq, auto* oo) {
      using T = std::remove_pointer_t<decltype(oo)>;
      auto with = [&](auto tiles, auto one_page, auto waves) {
        constexpr int WAVES = decltype(waves)::value;
        hipLaunchKernelGGL((cache_attn_kernel<N, BITS, decltype(tiles)::value,
                                              decltype(one_page)::value, WAVES, T>),
                           grid, dim3(WAVES * 64), 0, s, qq, c, a, oo);
      };
      auto run = [&](auto tiles, auto one_page) {
        constexpr int MANY = many_waves(N, BITS, decltype(tiles)::value);
        if (plan.many) with(tiles, one_page, std::integral_constant<int, MANY>{});
        else with(tiles, one_page, std::integral_constant<int, kAttnWaves>{});
      };
      auto by_page = [&](auto tiles) {
        if (c.lg_page >= 5) run(tiles, std::true_type{});
        else run(tiles, std::false_type{});
      };
      if constexpr (N <= 128) {
        if (ht == 2) by_page(std::integral_constant<int, 2>{});
      }
      if (ht == 1) by_page(std::integral_constant<int, 1>{});
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || a.slices == 1) return e;
      hipLaunchKernelGGL((cache_combine_kernel<N, T>),
                         dim3(static_cast<unsigned>(q_heads), static_cast<unsigned>(B)),
                         dim3(kAttnThreads), 0, s, a, oo);
      return hipGetLastError();
    };
    if (dt == Dt::F32) return go(static_cast<const float*>(q), static_cast<float*>(out));
    return go(static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out));
  });
}

}  // namespace qwha
