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

// ---- tokens as rows of the matrix instruction, staged by each wave for itself
// in LDS: 128-byte lines in, operands out. A chunk is 32 S columns of 16 rows;
// 16-byte piece p of row m lies at piece p ^ (m % pieces) of its row, so that
// the rows one read covers hit distinct banks.
template <typename T>
struct Rows;
template <>
struct Rows<uint16_t> {
  static constexpr int TOK = 16;     // tokens per 16 rows
};
// fp32 tokens: rows 4i .. 4i + 2 are a token's upper, middle and lower 8 bits
// of mantissa (each what is left of x after the one before, cut to bf16:
// exact), row 4i + 3 is zero. The three results of a token lie in one lane.
template <>
struct Rows<float> {
  static constexpr int TOK = 4;
};

template <int S>
struct Stage {
  static constexpr int PIECES = 4 * S;                 // of 16 bytes, per row
  static constexpr int WORDS = 16 * 16 * S;            // of 4 bytes, per 16 rows
  static __device__ __forceinline__ int at(int row, int piece) {
    return (row * PIECES + (piece ^ (row % PIECES))) * 4;
  }
};

// A wave's part of a chunk on its way from memory to LDS.
template <int S, typename T>
struct Incoming;
template <int S>
struct Incoming<S, uint16_t> {
  uint4 v[S];
  __device__ __forceinline__ void load(const uint16_t* x, int64_t K, int t0, int tokens, int col,
                                       int lane) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = i * 64 + lane, row = e / (4 * S), piece = e % (4 * S);
      v[i] = t0 + row < tokens
                 ? *reinterpret_cast<const uint4*>(x + (t0 + row) * K + col + 8 * piece)
                 : uint4{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void store(uint32_t* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = i * 64 + lane;
      *reinterpret_cast<uint4*>(lds + Stage<S>::at(e / (4 * S), e % (4 * S))) = v[i];
    }
  }
};
template <int S>
struct Incoming<S, float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* x, int64_t K, int t0, int tokens, int col,
                                       int lane) {
    const int tok = lane / (4 * S), piece = lane % (4 * S);   // lanes past 16 S have no piece
    const bool live = tok < 4 && t0 + tok < tokens;
    const float4* p = reinterpret_cast<const float4*>(x + (live ? (t0 + tok) * K + col + 8 * piece : 0));
    const float4 zero = float4{0.f, 0.f, 0.f, 0.f};
    v[0] = live ? p[0] : zero;
    v[1] = live ? p[1] : zero;
  }
  __device__ __forceinline__ void store(uint32_t* lds, int lane) const {
    const int tok = lane / (4 * S), piece = lane % (4 * S);
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t h[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[0][i] = __float_as_uint(f[i]);
      const float r1 = f[i] - __uint_as_float(h[0][i] & 0xFFFF0000u);
      h[1][i] = __float_as_uint(r1);
      h[2][i] = __float_as_uint(r1 - __uint_as_float(h[1][i] & 0xFFFF0000u));
    }
    if (tok < 4) {
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        uint32_t d[4] = {0u, 0u, 0u, 0u};
        if (part < 3)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] = __builtin_amdgcn_perm(h[part][2 * i + 1], h[part][2 * i], 0x07060302u);
        *reinterpret_cast<uint4*>(lds + Stage<S>::at(4 * tok + part, piece)) =
            uint4{d[0], d[1], d[2], d[3]};
      }
    }
  }
};

// ---- the transform of the tokens, zt[column][tp] fp32: four tokens of a
// block side by side in a workgroup, so that a column's values leave together
template <int LOG_N>
struct Zt {
  using F = Fwht<LOG_N>;
  static constexpr int TT = LOG_N <= 12 ? 4 : LOG_N == 13 ? 2 : 1;     // tokens side by side
  static constexpr int BLOCK = F::TPR * TT > 256 ? F::TPR * TT : 256;
  static constexpr int BLKS = BLOCK / (F::TPR * TT);                   // blocks of columns
};
template <int LOG_N, typename TIn>
__global__ __launch_bounds__(Zt<LOG_N>::BLOCK) void decode_fwht_kernel(const TIn* __restrict__ x,
                                                                       int tokens, int nblk,
                                                                       int tp,
                                                                       float* __restrict__ zt) {
  using F = Fwht<LOG_N>;
  using Z = Zt<LOG_N>;
  __shared__ float lds_all[Z::BLKS * Z::TT * F::LDS];
  const int slot = threadIdx.x / F::TPR, u = threadIdx.x % F::TPR;
  const int blk = blockIdx.x * Z::BLKS + slot / Z::TT, t = blockIdx.y * Z::TT + slot % Z::TT;
  const int64_t K = static_cast<int64_t>(nblk) << LOG_N;
  float* lds = lds_all + slot * F::LDS;
  float v[16];
  if (blk < nblk && t < tokens) {
    load16(x + t * K + (static_cast<int64_t>(blk) << LOG_N) + u * 16, v);
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = 0.f;
  }
  F::run(v, lds, u);
  constexpr float scale = 1.f / static_cast<float>(F::N);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 16; ++r) lds[F::pad(F::out_index(u, r))] = v[r] * scale;
  __syncthreads();
  const int b0 = blockIdx.x * Z::BLKS, t0 = blockIdx.y * Z::TT;
  for (int e = threadIdx.x; e < Z::BLKS * F::N; e += Z::BLOCK) {
    const int bl = e >> LOG_N, j = e & (F::N - 1);
    if (b0 + bl >= nblk) break;
    const float* src = lds_all + bl * Z::TT * F::LDS + F::pad(j);
    float* dst = zt + ((static_cast<int64_t>(b0 + bl) << LOG_N) + j) * tp + t0;
    if constexpr (Z::TT == 4) {
      *reinterpret_cast<float4*>(dst) =
          float4{src[0], src[F::LDS], src[2 * F::LDS], src[3 * F::LDS]};
    } else {
#pragma unroll
      for (int i = 0; i < Z::TT; ++i) dst[i] = src[i * F::LDS];
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
// The nonzeros of the same rows of F lie side by side in E and c: the first
// kEntries of them are fetched beside the codes and wait in LDS, so that only
// the gather of z is left behind the product.
struct DecodeArgs {
  int tokens, K, N, tp;
  QuantW qw;
  const float* zt;             // null without an adapter
  const int32_t* row_ptr;
  const int32_t* E;
  const float* c;
  float alpha;
};

constexpr int kThreads = kDecodeWaves * 64;
constexpr int kEntries = 4 * kThreads;   // nonzeros staged at a time

template <int BITS, int S, int MT, int NT, typename T>
__global__ __launch_bounds__(kThreads) void decode_kernel(const T* __restrict__ x, DecodeArgs a,
                                                          T* __restrict__ y) {
  constexpr int TB = Rows<T>::TOK * MT;              // tokens of the workgroup
  constexpr int U = 16 / S / MT > 0 ? 16 / S / MT : 1;
  constexpr int LD = 16 * NT + 1;
  constexpr int RPW = 2 * NT;                        // rows of F per wave
  constexpr int XW = MT * Stage<S>::WORDS;           // staged words of a wave
  constexpr int RW = TB * LD;                        // words of a wave's sums
  // a wave's staged tokens and, later, its sums share their place
  constexpr int WAVE = (XW > RW ? XW : RW) + 3 & ~3;
  __shared__ __attribute__((aligned(16))) uint32_t own[kDecodeWaves][WAVE];
  __shared__ float ad[16 * NT][TB + 4];
  __shared__ uint2 ent[kEntries];                    // column, value
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, t0 = blockIdx.y * TB;
  const int nchunks = a.K / (32 * S);

  int rp[RPW + 1], k0 = 0, kend = 0;
  if (a.zt != nullptr) {
    k0 = a.row_ptr[n0];
    kend = a.row_ptr[min(n0 + 16 * NT, a.N)];
#pragma unroll
    for (int i = 0; i <= RPW; ++i) rp[i] = a.row_ptr[min(n0 + w * RPW + i, a.N)];
  }

  const uint32_t* crow[NT];
  const float *srow[NT], *zrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(n0 + j * 16 + lr, a.N - 1);   // rows past N repeat the last
    crow[j] = a.qw.codes + n * a.qw.wpr;
    srow[j] = a.qw.scales + n * a.qw.gpr;
    zrow[j] = a.qw.zeros + n * a.qw.gpr;
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

  uint2 en[4];
  bool first = true;
  for (int c0 = w; c0 < nchunks || first; c0 += kDecodeWaves * U) {
    Codes<BITS, S> cw[U][NT];
    Incoming<S, T> xr[U][MT];
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
        xr[u][i].load(x, a.K, t0 + i * Rows<T>::TOK, a.tokens, col, lane);
    }
    if (first) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = static_cast<int64_t>(k0) + i * kThreads + threadIdx.x;
        if (k < kend) en[i] = uint2{static_cast<uint32_t>(a.E[2 * k + 1]), __float_as_uint(a.c[k])};
      }
      first = false;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u * kDecodeWaves >= nchunks) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) xr[u][i].store(&own[w][i * Stage<S>::WORDS], lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      f32x4 g[MT][NT], xs[MT];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        bf16x8 xf[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          xf[i] = *reinterpret_cast<const bf16x8*>(
              &own[w][i * Stage<S>::WORDS + Stage<S>::at(lr, lq * S + s)]);
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
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
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
  float* red = reinterpret_cast<float*>(own[w]);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) red[(i * 16 + 4 * lq + r) * LD + j * 16 + lr] = acc[i][j][r];
      } else {
        red[(i * 4 + lq) * LD + j * 16 + lr] = acc[i][j][0] + acc[i][j][1] + acc[i][j][2];
      }
    }

  // the nonzeros, a wave RPW rows: lpn lanes hold 4 tokens each of one
  // nonzero's column
  if (a.zt != nullptr) {
    const int lpn = min(a.tp, TB) / 4, npw = 64 / lpn;
    const int sub = lane / lpn;
    const float* zl = a.zt + t0 + (lane % lpn) * 4;
    f32x4 s4[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i) s4[i] = zero4;
    for (int kb = k0;;) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * kThreads + static_cast<int>(threadIdx.x) < kend - kb)
          ent[i * kThreads + threadIdx.x] = en[i];
      __syncthreads();
      const int held = min(kend - kb, kEntries);
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const int e1 = min(rp[i + 1] - kb, held);
#pragma unroll 4
        for (int k = max(rp[i] - kb, 0) + sub; k < e1; k += npw) {
          const uint2 e = ent[k];
          const f32x4 zv = *reinterpret_cast<const f32x4*>(zl + static_cast<int64_t>(e.x) * a.tp);
          const float cv = __uint_as_float(e.y);
#pragma unroll
          for (int r = 0; r < 4; ++r) s4[i][r] = fmaf(cv, zv[r], s4[i][r]);
        }
      }
      if (held == kend - kb) break;
      kb += held;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = static_cast<int64_t>(kb) + i * kThreads + threadIdx.x;
        if (k < kend) en[i] = uint2{static_cast<uint32_t>(a.E[2 * k + 1]), __float_as_uint(a.c[k])};
      }
    }
    for (int o = lpn; o < 64; o <<= 1)
#pragma unroll
      for (int i = 0; i < RPW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) s4[i][r] += __shfl_xor(s4[i][r], o);
    if (lane < lpn)
#pragma unroll
      for (int i = 0; i < RPW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) ad[w * RPW + i][lane * 4 + r] = s4[i][r];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < TB * 16 * NT; e += kThreads) {
    const int t = e / (16 * NT), n = e % (16 * NT);
    if (t0 + t >= a.tokens || n0 + n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) v += __uint_as_float(own[i][t * LD + n]);
    if (a.zt != nullptr) v = fmaf(a.alpha, ad[n][t], v);
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
  if (tiles == 1)
    return a.N >= 8192 ? decode_t<BITS, S, 1, 2, T>(x, a, y, s)
                       : decode_t<BITS, S, 1, 1, T>(x, a, y, s);
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
  using Z = Zt<LOG_N>;
  const dim3 grid((nblk + Z::BLKS - 1) / Z::BLKS, (tokens + Z::TT - 1) / Z::TT);
  hipLaunchKernelGGL((decode_fwht_kernel<LOG_N, T>), grid, dim3(Z::BLOCK), 0, s, x, tokens, nblk,
                     tp, zt);
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

// tokens a column of zt holds: a power of two, 4 at least
int padded_tokens(int T) {
  int tp = 4;
  while (tp < T) tp *= 2;
  return tp;
}

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
