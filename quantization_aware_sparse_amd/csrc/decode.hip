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

// (x & mask) | bits in one instruction: the mask in a vector register (one
// scalar operand per instruction), the bits a scalar
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(d) : "v"(x), "v"(mask), "s"(bits));
  return d;
}
__device__ __forceinline__ uint32_t in_vgpr(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Loads from a base that is the same in the whole wave plus 32-bit offsets
// (bytes) of the lanes: one address register a lane, none per load.
template <typename V>
__device__ __forceinline__ V ld_at(const void* base, uint32_t off) {
  return *reinterpret_cast<const V*>(static_cast<const char*>(base) + off);
}

// ---- a lane's codes of a chunk: 8 S consecutive columns of one row, as S
// operands of 8 columns each (bf16 of OFF + q, two to a word). `base` is the
// first row of the tile, `off` the lane's row in bytes, `col` the lane's first
// column (chunk plus `part`); MASK selects a code in both halves of a word.
template <int BITS, int S>
struct Codes;

template <int S>
struct Codes<4, S> {
  static constexpr float OFF = 16.f;
  static constexpr uint32_t MASK = 0x00780078u;
  uint32_t w[S];
  __device__ __forceinline__ void load(const uint32_t* base, uint32_t off, int chunk, int part,
                                       int) {
    const uint32_t* b = base + chunk / 8;
    const uint32_t o = off + part / 2;
    if constexpr (S == 4) {
      const uint4 v = ld_at<uint4>(b, o);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (S == 2) {
      const uint2 v = ld_at<uint2>(b, o);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = ld_at<uint32_t>(b, o);
    }
  }
  // bf16(16 + q) = 0x4180 | q << 3: low nibbles from w << 3, high ones from
  // w >> 1, a byte of each to a pair
  __device__ __forceinline__ bf16x8 operand(int i, uint32_t mask) const {
    const uint32_t u = w[i] << 3, v = w[i] >> 1;
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      d[k] = and_or(__builtin_amdgcn_perm(v, u, 0x0C040C00u + 0x00010001u * k), mask, 0x41804180u);
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

template <int S>
struct Codes<2, S> {
  static constexpr float OFF = 4.f;
  static constexpr uint32_t MASK = 0x00600060u;
  uint32_t w[S == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const uint32_t* base, uint32_t off, int chunk, int part,
                                       int) {
    const uint32_t* b = base + chunk / 16;
    const uint32_t o = off + part / 4;
    if constexpr (S == 4) {
      const uint2 v = ld_at<uint2>(b, o);
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (S == 2) {
      w[0] = ld_at<uint32_t>(b, o);
    } else {
      w[0] = ld_at<uint16_t>(b, o);
    }
  }
  // bf16(4 + q) = 0x4080 | q << 5
  __device__ __forceinline__ bf16x8 operand(int i, uint32_t mask) const {
    const uint32_t x = w[i / 2] >> (16 * (i % 2));
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      d[2 * k] = and_or(__builtin_amdgcn_perm(x << 3, x << 5, 0x0C040C00u + 0x00010001u * k),
                        mask, 0x40804080u);
      d[2 * k + 1] = and_or(__builtin_amdgcn_perm(x >> 1, x << 1, 0x0C040C00u + 0x00010001u * k),
                            mask, 0x40804080u);
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
  static constexpr uint32_t MASK = 0x00700070u;
  uint32_t w[NW];
  int sh;
  __device__ __forceinline__ void load(const uint32_t* base, uint32_t off, int chunk, int part,
                                       int wpr) {
    const int col = chunk + part, word = col / 10;
    sh = 3 * (col - 10 * word);
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = ld_at<uint32_t>(base, off + 4 * min(word + i, wpr - 1));
  }
  __device__ __forceinline__ uint32_t limb(int i) const {
    const uint32_t lo = (i < NW ? w[i] & 0x3FFFFFFFu : 0u) >> (2 * i);
    return lo | (i + 1 < NW ? w[i + 1] << (30 - 2 * i) : 0u);
  }
  // bf16(8 + q) = 0x4100 | q << 4
  __device__ __forceinline__ bf16x8 operand(int i, uint32_t mask) const {
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
      d[k] = and_or((t << 4) | (t << 17), mask, 0x41004100u);
    }
    bf16x8 r;
    __builtin_memcpy(&r, d, 16);
    return r;
  }
};

template <int S>
struct Codes<8, S> {
  static constexpr float OFF = 0.f;
  static constexpr uint32_t MASK = 0u;
  uint32_t w[2 * S];
  __device__ __forceinline__ void load(const uint32_t* base, uint32_t off, int chunk, int part,
                                       int) {
    const uint32_t* b = base + chunk / 4;
    const uint32_t o = off + part;
    if constexpr (S == 1) {
      const uint2 v = ld_at<uint2>(b, o);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < S / 2; ++i) {
        const uint4 v = ld_at<uint4>(b, o + 16 * i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  }
  // the upper halves of fp32(q): exact, q < 2^8
  __device__ __forceinline__ bf16x8 operand(int i, uint32_t) const {
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

// A wave's part of a chunk on its way from memory to LDS. Rows past the last
// token repeat it (their results are not stored).
template <int S, typename T>
struct Incoming;
template <int S>
struct Incoming<S, uint16_t> {
  uint4 v[S];
  // byte offsets of a lane's pieces in x
  static __device__ __forceinline__ void offsets(uint32_t* off, int K, int t0, int tokens,
                                                 int lane) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int e = i * 64 + lane;
      off[i] = 2 * (min(t0 + e / (4 * S), tokens - 1) * K + 8 * (e % (4 * S)));
    }
  }
  __device__ __forceinline__ void load(const uint16_t* x, const uint32_t* off) {
#pragma unroll
    for (int i = 0; i < S; ++i) v[i] = ld_at<uint4>(x, off[i]);
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
  static __device__ __forceinline__ void offsets(uint32_t* off, int K, int t0, int tokens,
                                                 int lane) {
    // lanes past 16 S have no piece of their own
    off[0] = 4 * (min(t0 + lane / (4 * S), tokens - 1) * K + 8 * (lane % (4 * S)));
  }
  __device__ __forceinline__ void load(const float* x, const uint32_t* off) {
    v[0] = ld_at<float4>(x, off[0]);
    v[1] = ld_at<float4>(x, off[0] + 16);
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
// With few tokens every workgroup transforms them itself, in LDS, while its
// codes are on their way (LOCAL): one launch, and no way through memory for z.
// The code is kept short (loops, no peeled copies): a workgroup runs through
// most of it once, and fetching instructions costs as much as fetching codes.
struct DecodeArgs {
  int tokens, K, N, tp;
  QuantW qw;
  const float* zt;             // zt[column][tp], unless LOCAL or p = 0
  const int32_t* row_ptr;      // null without an adapter
  const int32_t* E;
  const float* c;
  float alpha;                 // LOCAL: alpha / b, for the plain sums of the transform
  int log_b;
};

constexpr int kThreads = kDecodeWaves * 64;
constexpr int kEntries = 4 * kThreads;   // nonzeros staged at a time
constexpr int kLocal = 16384;            // T * K of tokens transformed in LDS
constexpr int kLocalTokens = 4;

__device__ __forceinline__ int zpad(int j) { return j + (j >> 4); }

// z <- x H per block of 2^log_b columns, z[t * zld + zpad(column)], unscaled:
// passes of 4 index bits, 16 values a thread, in place.
template <typename T>
__device__ __forceinline__ void local_transform(const T* __restrict__ x, int tokens, int K,
                                                int log_b, int zld, float* z) {
  const int per = K >> 4, items = tokens * per;
  int done = 0;                              // index bits done
#pragma unroll 1
  for (int lo = 0; done < log_b; lo = min(lo + 4, log_b - 4)) {
    const int hi = lo + 4;
#pragma unroll 1
    for (int e = threadIdx.x; e < items; e += kThreads) {
      const int t = e / per, u = e - t * per;
      const int j0 = (u & ((1 << lo) - 1)) | ((u >> lo) << hi);
      float* zr = z + t * zld;
      float v[16];
      if (done == 0) {
        load16(x + static_cast<int64_t>(t) * K + u * 16, v);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = zr[zpad(j0 + (r << lo))];
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (lo + b < done) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (r & (1 << b)) continue;
          const float p = v[r], q = v[r + (1 << b)];
          v[r] = p + q;
          v[r + (1 << b)] = p - q;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) zr[zpad(j0 + (r << lo))] = v[r];
    }
    done = hi;
    __syncthreads();
  }
}

template <int BITS, int S, int MT, int NT, typename T, bool LOCAL>
__global__ __launch_bounds__(kThreads) void decode_kernel(const T* __restrict__ x, DecodeArgs a,
                                                          T* __restrict__ y) {
  constexpr int TB = Rows<T>::TOK * MT;              // tokens of the workgroup
  constexpr int U = 16 / S / MT > 0 ? (16 / S / MT > 4 ? 4 : 16 / S / MT) : 1;
  constexpr int LD = 16 * NT + 1;
  constexpr int RPW = 2 * NT;                        // rows of F per wave
  constexpr int XW = MT * Stage<S>::WORDS;           // staged words of a wave
  constexpr int RW = TB * LD;                        // words of a wave's sums
  // a wave's staged tokens and, later, its sums share their place
  constexpr int WAVE = ((XW > RW ? XW : RW) + 3) & ~3;
  constexpr int XO = sizeof(T) == 2 ? S : 1;
  using Code = Codes<BITS, S>;
  __shared__ __attribute__((aligned(16))) uint32_t own[kDecodeWaves][WAVE];
  __shared__ float ad[16 * NT][LOCAL ? 4 : TB + 4];
  __shared__ uint2 ent[kEntries];                    // column, value
  extern __shared__ float zl[];                      // LOCAL: [tokens][zpad(K)]
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, t0 = blockIdx.y * TB;
  const int nchunks = a.K / (32 * S);
  const bool adapter = a.row_ptr != nullptr;

  int k0 = 0, kend = 0;
  if (adapter) {
    k0 = a.row_ptr[n0];
    kend = a.row_ptr[min(n0 + 16 * NT, a.N)];
  }
  const uint32_t* ctile = a.qw.codes + static_cast<int64_t>(n0) * a.qw.wpr;
  const float* stile = a.qw.scales + static_cast<int64_t>(n0) * a.qw.gpr;
  const float* ztile = a.qw.zeros + static_cast<int64_t>(n0) * a.qw.gpr;
  uint32_t coff[NT], soff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = min(j * 16 + lr, a.N - 1 - n0);       // rows past N repeat the last
    coff[j] = 4u * n * a.qw.wpr;
    soff[j] = 4u * n * a.qw.gpr;
  }
  uint32_t xoff[MT][XO];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    Incoming<S, T>::offsets(xoff[i], a.K, t0 + i * Rows<T>::TOK, a.tokens, lane);
  bf16x8 ones;
  {
    const uint32_t o[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    __builtin_memcpy(&ones, o, 16);
  }
  const uint32_t mask = in_vgpr(Code::MASK);
  const f32x4 zero4 = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = zero4;

  uint2 en[4];
  int rp[RPW + 1];
  int first = 1;
  int c0 = w;
#pragma unroll 1
  do {
    Code cw[U][NT];
    Incoming<S, T> xr[U][MT];
    float sc[U][NT], zo[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = min(c0 + u * kDecodeWaves, nchunks - 1) * 32 * S;   // in bounds past the end
      const int g = col >> a.qw.lg_group;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        cw[u][j].load(ctile, coff[j], col, 8 * S * lq, a.qw.wpr);
        sc[u][j] = ld_at<float>(stile + g, soff[j]);
        zo[u][j] = ld_at<float>(ztile + g, soff[j]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) xr[u][i].load(x + col, xoff[i]);
    }
    asm volatile("" : "+s"(first));     // no peeled copy of the loop for the first turn
    if (first) {
      first = 0;
      if (adapter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = min(i * kThreads + static_cast<int>(threadIdx.x), kend - k0 - 1);
          if (k >= 0) {
            const int64_t at = static_cast<int64_t>(k0) + k;
            en[i] = uint2{static_cast<uint32_t>(a.E[2 * at + 1]), __float_as_uint(a.c[at])};
          }
        }
#pragma unroll
        for (int i = 0; i <= RPW; ++i) rp[i] = a.row_ptr[min(n0 + w * RPW + i, a.N)];
        if constexpr (LOCAL) {
          const int zld = zpad(a.K);
          local_transform(x, a.tokens, a.K, a.log_b, zld, zl);
        }
      }
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
          const bf16x8 wf = cw[u][j].operand(s, mask);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            g[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], wf, s ? g[i][j] : zero4, 0, 0, 0);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float z = Code::OFF + zo[u][j];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = fmaf(sc[u][j], fmaf(-z, xs[i][r], g[i][j][r]), acc[i][j][r]);
      }
    }
    c0 += kDecodeWaves * U;
  } while (c0 < nchunks);
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
  // nonzero's column (LOCAL: one lane, its tokens one after the other)
  if (adapter) {
    const int lpn = LOCAL ? 1 : min(a.tp, TB) / 4, npw = 64 / lpn;
    const int sub = lane / lpn;
    const float* zg = a.zt + t0 + (lane % lpn) * 4;
    const int zld = zpad(a.K);
    f32x4 s4[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i) s4[i] = zero4;
    int kb = k0;
#pragma unroll 1
    for (;;) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ent[i * kThreads + threadIdx.x] = en[i];
      __syncthreads();
      const int held = min(kend - kb, kEntries);
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const int e1 = min(rp[i + 1] - kb, held);
#pragma unroll 2
        for (int k = max(rp[i] - kb, 0) + sub; k < e1; k += npw) {
          const uint2 e = ent[k];
          const float cv = __uint_as_float(e.y);
          if constexpr (LOCAL) {
            const float* zr = zl + zpad(e.x);
#pragma unroll
            for (int r = 0; r < kLocalTokens; ++r)
              if (r < a.tokens) s4[i][r] = fmaf(cv, zr[r * zld], s4[i][r]);
          } else {
            const f32x4 zv = *reinterpret_cast<const f32x4*>(zg + static_cast<int64_t>(e.x) * a.tp);
#pragma unroll
            for (int r = 0; r < 4; ++r) s4[i][r] = fmaf(cv, zv[r], s4[i][r]);
          }
        }
      }
      if (held == kend - kb) break;
      kb += held;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at =
            static_cast<int64_t>(kb) + min(i * kThreads + static_cast<int>(threadIdx.x), kend - kb - 1);
        en[i] = uint2{static_cast<uint32_t>(a.E[2 * at + 1]), __float_as_uint(a.c[at])};
      }
    }
#pragma unroll 1
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
#pragma unroll 1
  for (int e = threadIdx.x; e < TB * 16 * NT; e += kThreads) {
    const int t = e / (16 * NT), n = e % (16 * NT);
    if (t0 + t >= a.tokens || n0 + n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) v += __uint_as_float(own[i][t * LD + n]);
    if (adapter) v = fmaf(a.alpha, ad[n][t], v);
    Elem<T>::st(y, static_cast<int64_t>(t0 + t) * a.N + n0 + n, v);
  }
}

template <int BITS, int S, int MT, int NT, typename T, bool LOCAL>
hipError_t decode_t(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  constexpr int TB = Rows<T>::TOK * MT;
  const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (a.tokens + TB - 1) / TB);
  const size_t lds = LOCAL ? static_cast<size_t>(a.tokens) * (a.K + a.K / 16) * 4 : 0;
  hipLaunchKernelGGL((decode_kernel<BITS, S, MT, NT, T, LOCAL>), grid, dim3(kThreads), lds, s, x, a,
                     y);
  return hipGetLastError();
}

// tokens few enough for the transform in LDS
bool is_local(int T, int K) { return T <= kLocalTokens && T * K <= kLocal; }

template <int BITS, int S, typename T>
hipError_t decode_s(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  if (a.row_ptr != nullptr && is_local(a.tokens, a.K))
    return decode_t<BITS, S, 1, 1, T, true>(x, a, y, s);
  const int tiles = (a.tokens + Rows<T>::TOK - 1) / Rows<T>::TOK;
  if (tiles == 1)
    return a.N >= 8192 ? decode_t<BITS, S, 1, 2, T, false>(x, a, y, s)
                       : decode_t<BITS, S, 1, 1, T, false>(x, a, y, s);
  if (tiles == 2) return decode_t<BITS, S, 2, 1, T, false>(x, a, y, s);
  return decode_t<BITS, S, 4, 1, T, false>(x, a, y, s);
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
  if (p == 0 || is_local(static_cast<int>(T), K)) return 0;
  return static_cast<size_t>(K) * padded_tokens(static_cast<int>(T)) * 4;
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
  a.zt = nullptr;
  a.row_ptr = p > 0 ? row_ptr : nullptr;
  a.E = E;
  a.c = c;
  a.alpha = alpha;
  a.log_b = log_n;
  const bool through_memory = p > 0 && !is_local(T, a.K);
  if (through_memory)
    a.zt = static_cast<float*>(scratch);
  else
    a.alpha = alpha / static_cast<float>(1 << log_n);
  auto go = [&](auto* xx, auto* yy) {
    if (through_memory) {
      const hipError_t e = fwht_d(xx, T, log_n, nblk, a.tp, static_cast<float*>(scratch), s);
      if (e != hipSuccess) return e;
    }
    return decode_d(xx, a, yy, s);
  };
  if (dt == Dt::F32) return go(static_cast<const float*>(x), static_cast<float*>(y));
  return go(static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y));
}

}  // namespace qwha
