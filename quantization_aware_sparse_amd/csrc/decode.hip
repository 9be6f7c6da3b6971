// The quantized layer for the few tokens of a decoding step (QWHA notes,
// papernotes.org, 损失函数 / 训练策略; gist.science summary §4):
//   y = x W_Q^T + alpha z F^T,  z = FWHT(x) / b,  T <= 64 tokens.
//
//   decode_fwht_kernel  z, transposed: zt[column][token], so that one nonzero
//                       of F finds its column's tokens side by side;
//   decode_kernel       the base product on the bf16 matrix cores, the codes
//                       read once, and the nonzeros of the same rows of F.
//
// The base product per group g of columns, with codes q and OFF = 2^bits:
//   sum_j x_j (q_j - z) s = s (sum_j x_j (OFF + q_j) - (OFF + z) sum_j x_j).
// OFF + q is a bf16 number whose bits are a constant or-ed with q shifted, so
// unpacking costs a byte permute and an and-or per pair of codes; the smallest
// such OFF keeps the cancellation of the two sums small. 8-bit codes fill
// bf16's 8 bits by themselves (OFF = 0). Products are exact in fp32; only the
// fp32 additions round. fp32 tokens enter as three bf16 rows that sum to x
// exactly (8 + 8 + 8 bits), which take otherwise idle rows of the matrix
// instruction's 16.
#include <type_traits>

#include "fwht_core.h"
#include "launch.h"

namespace qwha {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kDecodeWaves = 8;

// (x & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  return (x & mask) | bits;
}

// ---- a lane's codes of a chunk: 8 S consecutive columns of one row, as S
// operands of 8 columns each (bf16 of OFF + q, two to a word)
template <int BITS, int S>
struct Codes;

template <int S>
struct Codes<4, S> {
  static constexpr float OFF = 16.f;
  uint32_t w[S];
  __device__ __forceinline__ void load(const uint32_t* row, int col, int) {
    const uint32_t* p = row + col / 8;
    if constexpr (S == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (S == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *p;
    }
  }
  // bf16(16 + q) = 0x4180 | q << 3: low nibbles from w << 3, high ones from
  // w >> 1, a byte of each to a pair
  __device__ __forceinline__ bf16x8 operand(int i) const {
    const uint32_t u = w[i] << 3, v = w[i] >> 1;
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      d[k] = and_or(__builtin_amdgcn_perm(v, u, 0x0C040C00u + 0x00010001u * k), 0x00780078u,
                    0x41804180u);
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

template <int S>
struct Codes<2, S> {
  static constexpr float OFF = 4.f;
  uint32_t w[S == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const uint32_t* row, int col, int) {
    if constexpr (S == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(row + col / 16);
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (S == 2) {
      w[0] = row[col / 16];
    } else {
      w[0] = reinterpret_cast<const uint16_t*>(row)[col / 8];
    }
  }
  // bf16(4 + q) = 0x4080 | q << 5
  __device__ __forceinline__ bf16x8 operand(int i) const {
    const uint32_t x = w[i / 2] >> (16 * (i % 2));
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      d[2 * k] = and_or(__builtin_amdgcn_perm(x << 3, x << 5, 0x0C040C00u + 0x00010001u * k),
                        0x00600060u, 0x40804080u);
      d[2 * k + 1] = and_or(__builtin_amdgcn_perm(x >> 1, x << 1, 0x0C040C00u + 0x00010001u * k),
                            0x00600060u, 0x40804080u);
    }
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

// 3-bit codes, 10 to a word: the words' 30-bit contents joined to one string
// of bits, shifted so that the lane's first code is at bit 0
template <int S>
struct Codes<3, S> {
  static constexpr float OFF = 8.f;
  static constexpr int NW = S == 4 ? 5 : S == 2 ? 3 : 2;   // (9 + 8 S) / 10 words, rounded up
  static constexpr int NL = S == 4 ? 3 : S == 2 ? 2 : 1;   // 24 S bits
  uint32_t w[NW];
  int sh;
  __device__ __forceinline__ void load(const uint32_t* row, int col, int wpr) {
    const int base = col / 10;
    sh = 3 * (col - 10 * base);
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = row[min(base + i, wpr - 1)];
  }
  __device__ __forceinline__ uint32_t limb(int i) const {
    const uint32_t lo = (i < NW ? w[i] & 0x3FFFFFFFu : 0u) >> (2 * i);
    return lo | (i + 1 < NW ? w[i + 1] << (30 - 2 * i) : 0u);
  }
  // bf16(8 + q) = 0x4100 | q << 4
  __device__ __forceinline__ bf16x8 operand(int i) const {
    uint32_t m[NL + 1];
#pragma unroll
    for (int k = 0; k < NL; ++k) m[k] = __builtin_amdgcn_alignbit(limb(k + 1), limb(k), sh);
    m[NL] = 0u;
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int bit = 24 * i + 6 * k;
      const uint32_t t =
          __builtin_amdgcn_alignbit(m[bit / 32 + 1 < NL ? bit / 32 + 1 : NL], m[bit / 32], bit % 32) &
          63u;
      d[k] = and_or((t << 4) | (t << 17), 0x00700070u, 0x41004100u);
    }
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

template <int S>
struct Codes<8, S> {
  static constexpr float OFF = 0.f;
  uint32_t w[2 * S];
  __device__ __forceinline__ void load(const uint32_t* row, int col, int) {
    const uint32_t* p = row + col / 4;
    if constexpr (S == 1) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < S / 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  }
  // the upper halves of fp32(q): exact, q < 2^8
  __device__ __forceinline__ bf16x8 operand(int i) const {
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = w[2 * i + k / 2] >> (16 * (k % 2));
      const uint32_t a = __float_as_uint(static_cast<float>(x & 0xFFu));
      const uint32_t b = __float_as_uint(static_cast<float>((x >> 8) & 0xFFu));
      d[k] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

// ---- tokens as rows of the matrix instruction: lane l supplies row l % 16
template <typename T>
struct Rows;
template <>
struct Rows<uint16_t> {
  static constexpr int TOK = 16;     // tokens per 16 rows
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* x, int64_t at, bool live) {
    v = live ? *reinterpret_cast<const uint4*>(x + at) : uint4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ bf16x8 operand(int) const {
    bf16x8 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
  }
};
// Rows 4i .. 4i + 2 are a token's upper, middle and lower 8 bits of mantissa
// (each what is left of x after the one before, cut to bf16: exact), row
// 4i + 3 is zero. The three results of a token lie in one lane.
template <>
struct Rows<float> {
  static constexpr int TOK = 4;
  float4 v[2];
  __device__ __forceinline__ void load(const float* x, int64_t at, bool live) {
    const float4 zero = float4{0.f, 0.f, 0.f, 0.f};
    v[0] = live ? reinterpret_cast<const float4*>(x + at)[0] : zero;
    v[1] = live ? reinterpret_cast<const float4*>(x + at)[1] : zero;
  }
  __device__ __forceinline__ bf16x8 operand(int lane) const {
    const int part = lane & 3;
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t h[8], d[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(f[i]) & 0xFFFF0000u;
      const float r1 = f[i] - __uint_as_float(a);
      const uint32_t b = __float_as_uint(r1) & 0xFFFF0000u;
      const uint32_t c = __float_as_uint(r1 - __uint_as_float(b));
      h[i] = part == 0 ? a : part == 1 ? b : part == 2 ? c : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_perm(h[2 * i + 1], h[2 * i], 0x07060302u);
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

// ---- the transform of the tokens, zt[column][tp] fp32
template <int LOG_N, typename TIn, int TT>
__global__ __launch_bounds__((Fwht<LOG_N>::TPR > 256 ? Fwht<LOG_N>::TPR : 256)) void
decode_fwht_kernel(const TIn* __restrict__ x, int tokens, int nblk, int tp,
                   float* __restrict__ zt) {
  using F = Fwht<LOG_N>;
  constexpr int BLOCK = F::TPR > 256 ? F::TPR : 256, RPW = BLOCK / F::TPR;
  __shared__ float lds_all[RPW * F::LDS];
  const int slot = threadIdx.x / F::TPR, u = threadIdx.x % F::TPR;
  const int blk = blockIdx.x * RPW + slot, t0 = blockIdx.y * TT;
  const bool live = blk < nblk;
  const int64_t K = static_cast<int64_t>(nblk) << LOG_N;
  float v[TT][F::EPT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    if (live && t0 + i < tokens) {
      load16(x + (t0 + i) * K + (static_cast<int64_t>(blk) << LOG_N) + u * 16, v[i]);
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) v[i][r] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) F::run(v[i], lds_all + slot * F::LDS, u);
  if (!live) return;
  constexpr float scale = 1.f / static_cast<float>(F::N);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float* dst = zt + ((static_cast<int64_t>(blk) << LOG_N) + F::out_index(u, r)) * tp + t0;
    if constexpr (TT == 4) {
      *reinterpret_cast<float4*>(dst) =
          float4{v[0][r] * scale, v[1][r] * scale, v[2][r] * scale, v[3][r] * scale};
    } else {
      dst[0] = v[0][r] * scale;
    }
  }
}

// ---- the product
// A workgroup takes 16 NT rows of W and MT tiles of tokens; its waves take the
// chunks of 32 S columns in turn, U of them with all loads in flight at once,
// and add up their sums in LDS. Lane l holds row l % 16 of its tile of W and,
// of the tokens, row l % 16; both hold the columns 8 S (l / 16) .. + 8 S of the
// chunk, so a lane reads consecutive bytes of a row of codes and a chunk never
// crosses a group (32 S <= group). Results: lane l has W's row l % 16 and the
// token rows 4 (l / 16) .. + 4.
struct DecodeArgs {
  int tokens, K, N, tp;
  QuantW qw;
  const float* zt;             // null without an adapter
  const int32_t* row_ptr;
  const int32_t* E;
  const float* c;
  float alpha;
};

template <int BITS, int S, int MT, int NT, typename T>
__global__ __launch_bounds__(kDecodeWaves * 64) void decode_kernel(const T* __restrict__ x,
                                                                   DecodeArgs a,
                                                                   T* __restrict__ y) {
  constexpr int TB = Rows<T>::TOK * MT;              // tokens of the workgroup
  constexpr int U = 16 / S / MT > 0 ? 16 / S / MT : 1;
  constexpr int LD = 16 * NT + 1;
  __shared__ float red[kDecodeWaves][TB][LD];
  __shared__ float ad[16 * NT][TB + 4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, t0 = blockIdx.y * TB;
  const int nchunks = a.K / (32 * S);

  const uint32_t* crow[NT];
  const float *srow[NT], *zrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(n0 + j * 16 + lr, a.N - 1);   // rows past N repeat the last
    crow[j] = a.qw.codes + n * a.qw.wpr;
    srow[j] = a.qw.scales + n * a.qw.gpr;
    zrow[j] = a.qw.zeros + n * a.qw.gpr;
  }
  int64_t xat[MT];
  bool xlive[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int t = t0 + i * Rows<T>::TOK + lr / (16 / Rows<T>::TOK);
    xlive[i] = t < a.tokens && (sizeof(T) == 2 || (lr & 3) != 3);
    xat[i] = xlive[i] ? static_cast<int64_t>(t) * a.K : 0;
  }
  bf16x8 ones;
  {
    const uint32_t o[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    __builtin_memcpy(&ones, o, 16);
  }
  const f32x4 zero4 = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = zero4;

  for (int c0 = w; c0 < nchunks; c0 += kDecodeWaves * U) {
    Codes<BITS, S> cw[U][NT];
    Rows<T> xr[U][S][MT];
    float sc[U][NT], zo[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = min(c0 + u * kDecodeWaves, nchunks - 1) * 32 * S;   // in bounds past the end
      const int g = col >> a.qw.lg_group;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        cw[u][j].load(crow[j], col + 8 * S * lq, a.qw.wpr);
        sc[u][j] = srow[j][g];
        zo[u][j] = zrow[j][g];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int s = 0; s < S; ++s)
          xr[u][s][i].load(x, xat[i] + col + 8 * S * lq + 8 * s, xlive[i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u * kDecodeWaves >= nchunks) break;
      f32x4 g[MT][NT], xs[MT];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        bf16x8 xf[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          xf[i] = xr[u][s][i].operand(lane);
          xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], ones, s ? xs[i] : zero4, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const bf16x8 wf = cw[u][j].operand(s);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            g[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], wf, s ? g[i][j] : zero4, 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float z = Codes<BITS, S>::OFF + zo[u][j];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = fmaf(sc[u][j], fmaf(-z, xs[i][r], g[i][j][r]), acc[i][j][r]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) red[w][i * 16 + 4 * lq + r][j * 16 + lr] = acc[i][j][r];
      } else {
        red[w][i * 4 + lq][j * 16 + lr] = acc[i][j][0] + acc[i][j][1] + acc[i][j][2];
      }
    }

  // the nonzeros of these rows of F, a wave a row: TB / 4 lanes hold 4 tokens
  // each of one nonzero's column
  constexpr int LPN = TB / 4, NPW = 64 / LPN;
  if (a.zt != nullptr) {
    const int sub = lane / LPN;
    const float* zl = a.zt + t0 + (lane % LPN) * 4;
    for (int i = w; i < 16 * NT; i += kDecodeWaves) {
      f32x4 s4 = zero4;
      if (n0 + i < a.N) {
        const int k1 = a.row_ptr[n0 + i + 1];
        for (int k = a.row_ptr[n0 + i] + sub; k < k1; k += NPW) {
          const int64_t j = a.E[2 * static_cast<int64_t>(k) + 1];
          const f32x4 zv = *reinterpret_cast<const f32x4*>(zl + j * a.tp);
          const float cv = a.c[k];
#pragma unroll
          for (int r = 0; r < 4; ++r) s4[r] = fmaf(cv, zv[r], s4[r]);
        }
      }
#pragma unroll
      for (int o = LPN; o < 64; o <<= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r) s4[r] += __shfl_xor(s4[r], o);
      if (lane < LPN)
#pragma unroll
        for (int r = 0; r < 4; ++r) ad[i][lane * 4 + r] = s4[r];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < TB * 16 * NT; e += kDecodeWaves * 64) {
    const int t = e / (16 * NT), n = e % (16 * NT);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) v += red[i][t][n];
    if (a.zt != nullptr) v = fmaf(a.alpha, ad[n][t], v);
    if (t0 + t < a.tokens && n0 + n < a.N)
      Elem<T>::st(y, static_cast<int64_t>(t0 + t) * a.N + n0 + n, v);
  }
}

template <int BITS, int S, int MT, int NT, typename T>
hipError_t decode_t(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  constexpr int TB = Rows<T>::TOK * MT;
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.tokens + TB - 1) / TB);
  hipLaunchKernelGGL((decode_kernel<BITS, S, MT, NT, T>), grid, dim3(kDecodeWaves * 64), 0, s, x, a,
                     y);
  return hipGetLastError();
}

template <int BITS, int S, typename T>
hipError_t decode_s(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  const int tiles = (a.tokens + Rows<T>::TOK - 1) / Rows<T>::TOK;
  if (tiles == 1) return decode_t<BITS, S, 1, 1, T>(x, a, y, s);
  if (tiles == 2) return decode_t<BITS, S, 2, 1, T>(x, a, y, s);
  return decode_t<BITS, S, 4, 1, T>(x, a, y, s);
}

template <int BITS, typename T>
hipError_t decode_b(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  if (a.qw.lg_group == 5) return decode_s<BITS, 1, T>(x, a, y, s);
  if (a.qw.lg_group == 6) return decode_s<BITS, 2, T>(x, a, y, s);
  return decode_s<BITS, 4, T>(x, a, y, s);
}

template <typename T>
hipError_t decode_d(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  switch (a.qw.bits) {
    case 2: return decode_b<2, T>(x, a, y, s);
    case 3: return decode_b<3, T>(x, a, y, s);
    case 4: return decode_b<4, T>(x, a, y, s);
    case 8: return decode_b<8, T>(x, a, y, s);
    default: return hipErrorInvalidValue;
  }
}

template <int LOG_N, typename T>
hipError_t fwht_t(const T* x, int tokens, int nblk, int tp, float* zt, hipStream_t s) {
  using F = Fwht<LOG_N>;
  constexpr int BLOCK = F::TPR > 256 ? F::TPR : 256, RPW = BLOCK / F::TPR;
  const int gx = (nblk + RPW - 1) / RPW;
  if (tokens > 1)
    hipLaunchKernelGGL((decode_fwht_kernel<LOG_N, T, 4>), dim3(gx, (tokens + 3) / 4), dim3(BLOCK),
                       0, s, x, tokens, nblk, tp, zt);
  else
    hipLaunchKernelGGL((decode_fwht_kernel<LOG_N, T, 1>), dim3(gx, 1), dim3(BLOCK), 0, s, x,
                       tokens, nblk, tp, zt);
  return hipGetLastError();
}

template <typename T>
hipError_t fwht_d(const T* x, int tokens, int log_n, int nblk, int tp, float* zt, hipStream_t s) {
  switch (log_n) {
#define QWHA_CASE(L) \
  case L:            \
    return fwht_t<L, T>(x, tokens, nblk, tp, zt, s);
    QWHA_CASE(6) QWHA_CASE(7) QWHA_CASE(8) QWHA_CASE(9) QWHA_CASE(10) QWHA_CASE(11)
    QWHA_CASE(12) QWHA_CASE(13) QWHA_CASE(14)
#undef QWHA_CASE
    default:
      return hipErrorInvalidValue;
  }
}

// tokens a column of zt holds: whole workgroup tiles
int padded_tokens(int T) { return (T + 15) / 16 * 16 == 48 ? 64 : (T + 15) / 16 * 16; }

}  // namespace

size_t decode_scratch_bytes(int64_t T, int K, int64_t p) {
  return p > 0 ? static_cast<size_t>(K) * padded_tokens(static_cast<int>(T)) * 4 : 0;
}

hipError_t launch_decode(const void* x, Dt dt, int T, int log_n, int nblk, int N,
                         const QuantW& qw, int64_t p, const int32_t* row_ptr, const int32_t* E,
                         const float* c, float alpha, void* y, void* scratch, hipStream_t s) {
  DecodeArgs a;
  a.tokens = T;
  a.K = nblk << log_n;
  a.N = N;
  a.tp = padded_tokens(T);
  a.qw = qw;
  a.zt = p > 0 ? static_cast<float*>(scratch) : nullptr;
  a.row_ptr = row_ptr;
  a.E = E;
  a.c = c;
  a.alpha = alpha;
  auto go = [&](auto* xx, auto* yy) {
    if (a.zt != nullptr) {
      const hipError_t e = fwht_d(xx, T, log_n, nblk, a.tp, static_cast<float*>(scratch), s);
      if (e != hipSuccess) return e;
    }
    return decode_d(xx, a, yy, s);
  };
  if (dt == Dt::F32) return go(static_cast<const float*>(x), static_cast<float*>(y));
  return go(static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y));
}

}  // namespace qwha
