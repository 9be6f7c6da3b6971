// The quantized layer for the few tokens of a decoding step (QWHA notes,
// papernotes.org, 损失函数 / 训练策略; gist.science summary §4):
//   y = x W_Q^T + alpha z F^T,  z = FWHT(x) / b,  T <= 64 tokens.
//
//   decode_kernel       up to 16 bf16 or 4 fp32 tokens, more of them for layers of
//                       fewer rows: the base product on the bf16 matrix cores,
//                       K split over the waves of a workgroup; with few tokens
//                       also the nonzeros of the same rows of F, the tokens
//                       transformed by every workgroup for itself;
//   decode_wide_kernel  more tokens: 64 bf16 or 16 fp32 ones a workgroup, K split
//                       over workgroups, partial sums;
//   decode_finish_kernel  partial sums and the nonzeros of F added up.
// The codes are read and unpacked once per such tile of tokens (16 or 4, 64 or
// 16): of the calls with several tiles the later ones find them in the caches,
// where they fit.
// Measured (median device time of twelve runs; bytes that must move at the 4.9
// TB/s of a copy):
//   4096 x 4096,  4 bits, 1 token,   524288 nonzeros   9.9 us of 3.2, one launch;
//   4096 x 14336, 4 bits, 3 tokens,  1179648          13.2 + 8.9 us of 9.7;
//   14336 x 4096, 3 bits, 16 tokens, 1179648          18.3 + 12.8 us of 8.6;
//   8192 x 8192,  2 bits, 64 tokens, 1048576          27.6 + 20.8 us of 7.8.
// Where z goes through memory, the first workgroups of the product's launch
// write it, transposed (zt[column][token], so that one nonzero of F finds its
// column's tokens side by side): the product does not need it, the finishing
// pass does.
//
// The base product per group g of columns, with codes q and OFF = 2^bits:
//   sum_j x_j (q_j - z) s = s (sum_j x_j (OFF + q_j) - (OFF + z) sum_j x_j).
// OFF + q is a bf16 number whose bits are a constant or-ed with q shifted, so
// unpacking costs a byte permute and an and-or per pair of codes; the smallest
// such OFF keeps the cancellation of the two sums small. 8-bit codes fill
// bf16's 8 bits by themselves (OFF = 0). Products are exact in fp32; only the
// fp32 additions round. fp32 tokens enter as three bf16 rows that sum to x
// exactly (8 + 8 + 8 bits), which take otherwise idle rows of the matrix
// instruction's 16; the instruction takes numbers below 2^-126 as zeros.
#include <type_traits>

#include "fwht_core.h"
#include "launch.h"
#include "mfma_codes.h"

namespace qwha {

namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kDecodeWaves = 8;
constexpr int kThreads = kDecodeWaves * 64;
constexpr int kSpan = 128;      // columns of a span: 32 per quarter of the wave

// Loads from a base that is the same in the whole wave plus 32-bit offsets
// (bytes) of the lanes: one address register a lane, none per load.
template <typename V>
__device__ __forceinline__ V ld_at(const void* base, uint32_t off) {
  return *reinterpret_cast<const V*>(static_cast<const char*>(base) + off);
}

// ---- codes
// Lane l reads row l % 16 and, in quarter l / 16 of the wave, the 32 columns
// 32 (l / 16) .. of a span: 64 consecutive bytes of a row of 4-bit codes. They
// are four units of 8 columns, one per matrix instruction. The columns that
// one instruction adds up must share a group. Groups of 128 and more do; for
// smaller ones the units change places between quarters (an exchange of index
// bits, unit (a1 a0) of quarter (b1 b0)):
//   group 64:  a1 <-> b1: units 0 and 1 then hold the span's first group;
//   group 32:  and a0 <-> b0: unit i holds group i.
// unit_piece() is the piece of 8 columns that a unit then holds.
enum Mode { kWide = 0, kHalf = 1, kFull = 2 };    // group >= 128, 64, 32

template <int MODE>
__device__ __forceinline__ int unit_piece(int s, int q) {
  if (MODE == kWide) return 4 * q + s;
  if (MODE == kHalf) return 4 * (2 * (s >> 1) + (q & 1)) + 2 * (q >> 1) + (s & 1);
  return 4 * s + q;
}

// a's upper 32 lanes <-> b's lower ones; a's odd rows of 16 lanes <-> b's even
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int BITS>
struct Codes {
  static constexpr float OFF = BITS == 8 ? 0.f : static_cast<float>(1 << BITS);
  // a code in both halves of a word, where bf16(OFF + q) has it; OFF's bits
  static constexpr uint32_t MASK = BITS == 2 ? 0x00600060u : BITS == 3 ? 0x00700070u : 0x00780078u;
  static constexpr uint32_t BASE = BITS == 2 ? 0x40804080u : BITS == 3 ? 0x41004100u : 0x41804180u;
  static constexpr int UW = BITS == 8 ? 2 : 1;        // words per unit
  static constexpr int NW = BITS == 2 ? 2 : BITS == 8 ? 8 : 4;   // words read

  uint32_t w[NW];
  int sh;     // 3-bit codes

  // `base`: the tile's first row; `off`: the lane's row, in bytes; `col`: the
  // lane's first column, 32 columns inside the row
  __device__ __forceinline__ void load(const uint32_t* base, uint32_t off, int col) {
    if constexpr (BITS == 2) {
      const uint2 v = ld_at<uint2>(base, off + col / 4);
      w[0] = v.x; w[1] = v.y;
    } else if constexpr (BITS == 4) {
      const uint4 v = ld_at<uint4>(base, off + col / 2);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = ld_at<uint4>(base, off + col + 16 * i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    } else {
      // 10 codes to a word: col is a multiple of 32, so the 32 codes start at
      // an even one and lie in 4 words; the row has them, since for col = K - 32
      // floor((K - 32) / 10) + 4 = floor((K + 8) / 10) <= ceil(K / 10)
      const int word = col / 10;
      sh = 3 * (col - 10 * word);
      const u32x4_any v = ld_at<u32x4_any>(base, off + 4 * word);
      w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    }
  }

  // the four units, in place of the words
  template <int MODE>
  __device__ __forceinline__ void units(uint32_t (&u)[4][UW]) const {
    if constexpr (BITS == 2) {
      u[0][0] = w[0]; u[1][0] = w[0] >> 16; u[2][0] = w[1]; u[3][0] = w[1] >> 16;
    } else if constexpr (BITS == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i][0] = w[i];
    } else if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) { u[i][0] = w[2 * i]; u[i][1] = w[2 * i + 1]; }
    } else {
      // the words' 30-bit contents as one string of bits, from bit sh on
      const uint32_t l0 = (w[0] & 0x3FFFFFFFu) | (w[1] << 30);
      const uint32_t l1 = ((w[1] & 0x3FFFFFFFu) >> 2) | (w[2] << 28);
      const uint32_t l2 = ((w[2] & 0x3FFFFFFFu) >> 4) | (w[3] << 26);
      const uint32_t l3 = (w[3] & 0x3FFFFFFFu) >> 6;
      const uint32_t m0 = __builtin_amdgcn_alignbit(l1, l0, sh);
      const uint32_t m1 = __builtin_amdgcn_alignbit(l2, l1, sh);
      const uint32_t m2 = __builtin_amdgcn_alignbit(l3, l2, sh);
      u[0][0] = m0;                                        // 24 bits each
      u[1][0] = __builtin_amdgcn_alignbit(m1, m0, 24);
      u[2][0] = __builtin_amdgcn_alignbit(m2, m1, 16);
      u[3][0] = m2 >> 8;
    }
    if constexpr (MODE != kWide) {
#pragma unroll
      for (int i = 0; i < UW; ++i) {
        swap32(u[0][i], u[2][i]);
        swap32(u[1][i], u[3][i]);
        if constexpr (MODE == kFull) {
          swap16(u[0][i], u[1][i]);
          swap16(u[2][i], u[3][i]);
        }
      }
    }
  }

  // 8 codes as bf16(OFF + q), two to a word
  static __device__ __forceinline__ bf16x8 operand(const uint32_t (&u)[UW], uint32_t mask) {
    uint32_t d[4];
    if constexpr (BITS == 8) {
      return operand8(u[0], u[1]);
    } else if constexpr (BITS == 4) {
      return operand4(u[0], mask);
    } else if constexpr (BITS == 2) {
      const uint32_t a = u[0] << 5, b = u[0] << 3, c = u[0] << 1, e = u[0] >> 1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t sel = 0x0C040C00u + 0x00010001u * k;
        d[2 * k] = and_or(__builtin_amdgcn_perm(b, a, sel), mask, BASE);
        d[2 * k + 1] = and_or(__builtin_amdgcn_perm(e, c, sel), mask, BASE);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t t = (u[0] >> (6 * k)) & 63u;
        d[k] = and_or((t << 4) | (t << 17), mask, BASE);
      }
    }
    return as_operand(d);
  }
};

// ---- tokens, staged in LDS as rows of the matrix instruction
// A tile is 16 rows of a span; 16-byte piece p of row m lies at piece
// p ^ m of its row, so that the rows one read covers hit distinct banks.
constexpr int kTileWords = 16 * kSpan / 2;
__device__ __forceinline__ int tile_at(int row, int piece) { return row * 64 + ((piece ^ row) & 15) * 4; }

template <typename T>
struct Rows;
template <>
struct Rows<uint16_t> {
  static constexpr int TOK = 16;     // tokens per tile
};
// fp32 tokens: rows 4i .. 4i + 2 are a token's upper, middle and lower 8 bits
// of mantissa (each what is left of x after the one before, cut to bf16:
// exact), row 4i + 3 is zero. The three results of a token lie in one lane.
template <>
struct Rows<float> {
  static constexpr int TOK = 4;
};

// 8 columns of one token, between memory and LDS.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* x, uint32_t row_off, int col) {
    v = ld_at<uint4>(x, row_off + 2 * col);
  }
  __device__ __forceinline__ void store(uint32_t* tile, int tok, int piece) const {
    *reinterpret_cast<uint4*>(tile + tile_at(tok, piece)) = v;
  }
};
template <>
struct Piece<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* x, uint32_t row_off, int col) {
    v[0] = ld_at<float4>(x, row_off + 4 * col);
    v[1] = ld_at<float4>(x, row_off + 4 * col + 16);
  }
  __device__ __forceinline__ void store(uint32_t* tile, int tok, int piece) const {
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t h[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[0][i] = __float_as_uint(f[i]);
      const float r1 = f[i] - __uint_as_float(h[0][i] & 0xFFFF0000u);
      h[1][i] = __float_as_uint(r1);
      h[2][i] = __float_as_uint(r1 - __uint_as_float(h[1][i] & 0xFFFF0000u));
    }
#pragma unroll
    for (int part = 0; part < 4; ++part) {
      uint32_t d[4] = {0u, 0u, 0u, 0u};
      if (part < 3)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = __builtin_amdgcn_perm(h[part][2 * i + 1], h[part][2 * i], 0x07060302u);
      *reinterpret_cast<uint4*>(tile + tile_at(4 * tok + part, piece)) = uint4{d[0], d[1], d[2], d[3]};
    }
  }
};

struct DecodeArgs {
  int tokens, K, N, tp;
  int64_t p;
  QuantW qw;
  const float* zt;             // zt[column][tp], where z goes through memory
  const int32_t* row_ptr;      // null without an adapter
  const int32_t* E;
  const float* c;
  float alpha;                 // alpha / b for the plain sums of a transform in LDS
  int log_b;
  // partial sums, where a finishing pass follows: [slices][ceil(N / 16)][tokens]
  // [16], so that it reads the 16 rows it finishes as one run of memory
  float* part;
  int slices;
  float* z_out;                // zt, written by the launch's first z_blocks workgroups
  int z_cols, z_blocks;        // columns of a token that one of them transforms
};

// Steps and zeros of a span's groups for one row: G neighbours in memory.
template <int G>
struct Groups {
  float v[G];
  // `row`: the tile's first row, `off` the lane's row in bytes, `g` the span's
  // first group; where the row has fewer than G left, its last one repeats
  __device__ __forceinline__ void load(const float* row, uint32_t off, int g, int gpr) {
    if constexpr (G == 1) {
      v[0] = ld_at<float>(row + g, off);
    } else if (g + G <= gpr) {
      typedef float any __attribute__((ext_vector_type(G), aligned(4)));
      const any x = ld_at<any>(row + g, off);
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] = x[i];
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] = ld_at<float>(row + min(g + i, gpr - 1), off);
    }
  }
};

__device__ __forceinline__ int64_t part_at(const DecodeArgs& a, int slice, int t, int n) {
  const int64_t tiles = (a.N + 15) >> 4;
  return ((slice * tiles + (n >> 4)) * a.tokens + t) * 16 + (n & 15);
}

// The product of one span: acc += s (x (OFF + q) - (OFF + z) sum x), group by
// group. Lane l's results: W's row l % 16 of tile j and the token rows
// 4 (l / 16) .. + 4 of tile i.
template <int BITS, int MODE, int MT, int NT>
__device__ __forceinline__ void span_product(const uint32_t* tiles, const Codes<BITS> (&cw)[NT],
                                             const Groups<1 << MODE> (&sc)[NT],
                                             const Groups<1 << MODE> (&zo)[NT], bool half_span,
                                             uint32_t mask, bf16x8 ones, int lr, int lq,
                                             f32x4 (&acc)[MT][NT]) {
  using Code = Codes<BITS>;
  constexpr int G = 1 << MODE, PER = 4 / G;    // groups, instructions per group
  const f32x4 zero4 = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t u[NT][4][Code::UW];
#pragma unroll
  for (int j = 0; j < NT; ++j) cw[j].template units<MODE>(u[j]);
  f32x4 g[MT][NT], xs[MT];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (MODE != kWide && s == 2 && half_span) break;     // the columns end after two units
    bf16x8 xf[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      xf[i] = *reinterpret_cast<const bf16x8*>(tiles + i * kTileWords +
                                               tile_at(lr, unit_piece<MODE>(s, lq)));
      xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], ones, s % PER ? xs[i] : zero4, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const bf16x8 wf = Code::operand(u[j][s], mask);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        g[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], wf, s % PER ? g[i][j] : zero4, 0, 0, 0);
    }
    if (s % PER == PER - 1) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float z = Code::OFF + zo[j].v[s / PER];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = fmaf(sc[j].v[s / PER], fmaf(-z, xs[i][r], g[i][j][r]), acc[i][j][r]);
      }
    }
  }
}

__device__ __forceinline__ bf16x8 bf16_ones() {
  const uint32_t o[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  return as_operand(o);
}

// ---- the transform in LDS
__device__ __forceinline__ int zpad(int j) { return j + (j >> 4); }

// 16 consecutive values on their way
template <typename T>
struct Raw16;
template <>
struct Raw16<uint16_t> {
  uint4 v[2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    v[0] = reinterpret_cast<const uint4*>(p)[0];
    v[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
        f[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    }
  }
};
template <>
struct Raw16<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = v[i].x; f[4 * i + 1] = v[i].y; f[4 * i + 2] = v[i].z; f[4 * i + 3] = v[i].w;
    }
  }
};

__device__ __forceinline__ void butterflies(float* v, int b) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r & (1 << b)) continue;
    const float p = v[r], q = v[r + (1 << b)];
    v[r] = p + q;
    v[r + (1 << b)] = p - q;
  }
}

// z[t * zld + zpad(column)] <- x H per block of 2^log_b columns, unscaled:
// passes of 4 index bits, 16 values a thread, in place. `raw` holds the
// thread's first 16 values (fetched before anything else is waited for).
template <int THREADS, typename T>
__device__ __forceinline__ void local_transform(const T* __restrict__ x, Raw16<T> raw, int items,
                                                int per, int log_b, int zld, float* z) {
  float v[16];
#pragma unroll 1
  for (int e = threadIdx.x; e < items;) {
    raw.get(v);
    const int t = e / per, u = e - t * per;
    e += THREADS;
    if (e < items) raw.load(x + static_cast<int64_t>(e) * 16);
#pragma unroll
    for (int b = 0; b < 4; ++b) butterflies(v, b);
    float* zr = z + t * zld + 17 * u;
#pragma unroll
    for (int r = 0; r < 16; ++r) zr[r] = v[r];
  }
  __syncthreads();
#pragma unroll 1
  for (int done = 4; done < log_b; done += 4) {
    const int lo = min(done, log_b - 4);
#pragma unroll 1
    for (int e = threadIdx.x; e < items; e += THREADS) {
      const int t = e / per, u = e - t * per;
      float* zr = z + t * zld;
      const int j0 = (u & ((1 << lo) - 1)) | ((u >> lo) << (lo + 4));
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = zr[zpad(j0 + (r << lo))];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (lo + b >= done) butterflies(v, b);
#pragma unroll
      for (int r = 0; r < 16; ++r) zr[zpad(j0 + (r << lo))] = v[r];
    }
    __syncthreads();
  }
}

// zt[column][token] for z_cols columns (whole blocks) of one token: workgroup
// `block` of the launch. Workgroups go round the 8 XCDs in turn; those of one XCD
// take neighbouring tokens, whose values lie side by side, so that its L2 joins
// them before they go to memory.
template <int THREADS, typename T>
__device__ __forceinline__ void write_z(const T* __restrict__ x, const DecodeArgs& a, int block,
                                        float* lds) {
  const int each = a.z_blocks / 8, more = a.z_blocks % 8, xcd = block % 8;
  const int at = xcd * each + min(xcd, more) + block / 8;
  const int t = at % a.tokens, c0 = at / a.tokens * a.z_cols;
  const int cols = min(a.z_cols, a.K - c0), items = cols >> 4;
  const T* row = x + static_cast<int64_t>(t) * a.K + c0;
  Raw16<T> raw;
  raw.load(row + 16 * min(static_cast<int>(threadIdx.x), items - 1));
  local_transform<THREADS>(row, raw, items, items, a.log_b, zpad(cols), lds);
  const float scale = 1.f / static_cast<float>(1 << a.log_b);
  float* out = a.z_out + static_cast<int64_t>(c0) * a.tp + t;
  for (int j = threadIdx.x; j < cols; j += THREADS)
    out[static_cast<int64_t>(j) * a.tp] = lds[zpad(j)] * scale;
}

// ---- the nonzeros of some rows of F: side by side in E and c. The first
// kEntries of them are fetched beside whatever comes first and wait in LDS, so
// that only the gather of z is left; each further round's are fetched while the
// one before is worked on. 64 / RPW lanes take a row, or with SPLIT all waves one
// row, each its share.
constexpr int kEntriesEach = 8;                 // per thread: fewer rounds beat fewer registers
constexpr int kEntries = kEntriesEach * kThreads;
constexpr int kLocal = 4096, kLocalOne = 16384;  // T * K transformed in LDS; of one token
constexpr int kLocalTokens = 4;

struct Entries {
  uint2 e[kEntriesEach];                            // column, value
  __device__ __forceinline__ void load(const DecodeArgs& a, int kb, int kend) {
    if (kend <= kb) return;
#pragma unroll
    for (int i = 0; i < kEntriesEach; ++i) {
      const int64_t at =
          static_cast<int64_t>(kb) + min(i * kThreads + static_cast<int>(threadIdx.x), kend - kb - 1);
      e[i] = uint2{static_cast<uint32_t>(a.E[2 * at + 1]), __float_as_uint(a.c[at])};
    }
  }
  __device__ __forceinline__ void store(uint2* ent) const {
#pragma unroll
    for (int i = 0; i < kEntriesEach; ++i) ent[i * kThreads + threadIdx.x] = e[i];
  }
};

// Sums over the LANES lanes of a row that hold the same tokens: those that
// differ in the bits from `from` on. Within rows of 16 lanes through DPP.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, int from) {
  if (from <= 1) v += lane_xor<1>(v);
  if (from <= 2) v += lane_xor<2>(v);
  if (from <= 4) v += lane_xor<4>(v);
  if (from <= 8) v += lane_xor<8>(v);
  if constexpr (LANES > 16) {
    if (from <= 16) v += __shfl_xor(v, 16);
  }
  if constexpr (LANES > 32) {
    if (from <= 32) v += __shfl_xor(v, 32);
  }
  return v;
}

// ad[row][token] for the workgroup's 8 RPW rows (SPLIT: ad[wave][token], to be
// added up). LOCAL: z in LDS, a lane a nonzero, its tokens one after the other;
// else lpn lanes hold 4 tokens each of a nonzero's column. All threads call it.
template <int RPW, bool LOCAL, bool SPLIT, int LDA>
__device__ __forceinline__ void nonzeros(const DecodeArgs& a, Entries& en, uint2* ent, int k0,
                                         int kend, int beg, int end, int lpn, const float* zl,
                                         float (*ad)[LDA]) {
  constexpr int LPR = 64 / RPW;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int in_row = lane & (LPR - 1);
  const int npw = (SPLIT ? kDecodeWaves : 1) * (LPR / lpn);
  const int sub = in_row / lpn + (SPLIT ? w * (LPR / lpn) : 0);
  const float* zg = a.zt + (in_row & (lpn - 1)) * 4;
  const int zld = zpad(a.K);
  f32x4 s4 = f32x4{0.f, 0.f, 0.f, 0.f};
  int kb = k0;
#pragma unroll 1
  for (;;) {
    en.store(ent);
    __syncthreads();
    const int held = min(kend - kb, kEntries);
    const int e1 = min(end - kb, held);
    if (held < kend - kb) en.load(a, kb + held, kend);
#pragma clang loop unroll_count(LOCAL ? 2 : 8)
    for (int k = max(beg - kb, 0) + sub; k < e1; k += npw) {
      const uint2 e = ent[k];
      const float cv = __uint_as_float(e.y);
      if constexpr (LOCAL) {
        const float* zr = zl + zpad(e.x);
        s4[0] = fmaf(cv, zr[0], s4[0]);
        if (a.tokens > 1) {
#pragma unroll
          for (int r = 1; r < kLocalTokens; ++r)
            if (r < a.tokens) s4[r] = fmaf(cv, zr[r * zld], s4[r]);
        }
      } else {
        const f32x4 zv = *reinterpret_cast<const f32x4*>(zg + static_cast<int64_t>(e.x) * a.tp);
#pragma unroll
        for (int r = 0; r < 4; ++r) s4[r] = fmaf(cv, zv[r], s4[r]);
      }
    }
    if (held == kend - kb) break;
    kb += held;
    __syncthreads();
  }
  s4[0] = lanes_sum<LPR>(s4[0], lpn);
  if (a.tokens > 1)
#pragma unroll
    for (int r = 1; r < 4; ++r) s4[r] = lanes_sum<LPR>(s4[r], lpn);
  if (in_row < lpn)
#pragma unroll
    for (int r = 0; r < 4; ++r) ad[w * RPW + lane / LPR][in_row * 4 + r] = s4[r];
}

// ---- tiles of 16 bf16 or 4 fp32 tokens
// A workgroup takes 16 NT rows of W and a tile of tokens; its waves take the spans in turn, D of
// them on their way at any time, and add up their sums in LDS. The code is kept
// short (loops, no peeled copies): a workgroup runs through much of it once, and
// fetching instructions costs as much as fetching codes. FEW: at most 4 tokens,
// of whose tiles only the first 4 rows are staged (the others' results are not
// used, whatever they hold). LOCAL: every workgroup transforms the tokens for
// itself while its codes are on their way, and adds its rows of F: one launch,
// and no way through memory for z. Bound by latency: a start, the tokens' passes
// through LDS and the spans that 256 workgroups have in flight.
// With groups of 128 and more the rows' steps and zeros, one run of memory, are
// staged in LDS: read span by span they cost twice the codes' instructions, and
// it is the rate of such scattered reads that bounds the kernel.
template <int BITS, int MODE, int NT, typename T, bool FEW, bool LOCAL>
__global__ __launch_bounds__(kThreads) void decode_kernel(const T* __restrict__ x, DecodeArgs a,
                                                          T* __restrict__ y) {
  constexpr int TB = Rows<T>::TOK;
  constexpr int D = 4;                               // spans on their way
  constexpr int G = 1 << MODE;
  constexpr bool STAGED = MODE == kWide;             // steps and zeros in LDS
  constexpr int PX = sizeof(T) == 2 && !FEW ? 4 : 1; // pieces of a span per lane
  constexpr int RPW = 2 * NT;                        // rows of F per wave
  constexpr int LD = 16 * NT + 1;
  using Code = Codes<BITS>;
  __shared__ __attribute__((aligned(16))) uint32_t own[kDecodeWaves][kTileWords];
  __shared__ float ad[LOCAL ? 16 * NT : 1][LOCAL ? 8 : 1];
  __shared__ uint2 ent[LOCAL ? kEntries : 1];
  extern __shared__ __attribute__((aligned(16))) float dyn[];   // steps and zeros, then z
  if (static_cast<int>(blockIdx.x) < a.z_blocks) {
    write_z<kThreads>(x, a, blockIdx.x, dyn);
    return;
  }
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int tiles_n = (a.N + 16 * NT - 1) / (16 * NT), block = blockIdx.x - a.z_blocks;
  const int n0 = block % tiles_n * 16 * NT, t0 = LOCAL ? 0 : block / tiles_n * TB;
  const int spans = (a.K + kSpan - 1) / kSpan;
  const int rows = min(16 * NT, a.N - n0), toks = min(a.tokens - t0, TB);

  int k0 = 0, kend = 0, beg = 0, end = 0;
  Raw16<T> raw;
  if constexpr (LOCAL) {
    k0 = a.row_ptr[n0];
    kend = a.row_ptr[n0 + rows];
    const int row = n0 + w * RPW + lane / (64 / RPW);
    beg = a.row_ptr[min(row, a.N)];
    end = a.row_ptr[min(row + 1, a.N)];
    raw.load(x + 16 * min(static_cast<int>(threadIdx.x), (a.tokens * a.K >> 4) - 1));
  }
  const uint32_t* ctile = a.qw.codes + static_cast<int64_t>(n0) * a.qw.wpr;
  const float* stile = a.qw.scales + static_cast<int64_t>(n0) * a.qw.gpr;
  const float* ztile = a.qw.zeros + static_cast<int64_t>(n0) * a.qw.gpr;
  uint32_t coff[NT], soff[NT], xoff[PX];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = min(j * 16 + lr, rows - 1);           // rows past N repeat the last
    coff[j] = 4u * n * a.qw.wpr;
    soff[j] = STAGED ? n * (a.qw.gpr + 1) : 4u * n * a.qw.gpr;
  }
#pragma unroll
  for (int i = 0; i < PX; ++i)                          // tokens past the last repeat it
    xoff[i] = sizeof(T) * (t0 + min(4 * i + lq, toks - 1)) * a.K;

  struct Slot {
    Code cw[NT];
    Groups<G> sc[NT], zo[NT];
    Piece<T> xp[PX];
  } slot[D];
  auto fetch = [&](Slot& s, int span) {
    const int c0 = min(span, spans - 1) * kSpan;        // in bounds past the end
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      s.cw[j].load(ctile, coff[j], min(c0 + 32 * lq, a.K - 32));
      if constexpr (!STAGED) {
        s.sc[j].load(stile, soff[j], c0 >> a.qw.lg_group, a.qw.gpr);
        s.zo[j].load(ztile, soff[j], c0 >> a.qw.lg_group, a.qw.gpr);
      }
    }
#pragma unroll
    for (int i = 0; i < PX; ++i) s.xp[i].load(x, xoff[i], min(c0 + 8 * lr, a.K - 8));
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(slot[d], w + d * kDecodeWaves);
  // rows of gpr steps, padded by one, and as many zeros
  float* steps = dyn;
  float* zeros = dyn + 16 * NT * (a.qw.gpr + 1);
  if constexpr (STAGED) {
#pragma unroll 1
    for (int r = w; r < rows; r += kDecodeWaves)
      for (int g = lane; g < a.qw.gpr; g += 64) {
        steps[r * (a.qw.gpr + 1) + g] = stile[r * a.qw.gpr + g];
        zeros[r * (a.qw.gpr + 1) + g] = ztile[r * a.qw.gpr + g];
      }
  }
  float* zl = dyn + (STAGED ? 32 * NT * (a.qw.gpr + 1) : 0);   // LOCAL: [tokens][zpad(K)]
  Entries en;
  if constexpr (LOCAL) {
    en.load(a, k0, kend);
    local_transform<kThreads>(x, raw, a.tokens * a.K >> 4, a.K >> 4, a.log_b, zpad(a.K), zl);
  } else if constexpr (STAGED) {
    __syncthreads();
  }

  const uint32_t mask = in_vgpr(Code::MASK);
  const bf16x8 ones = bf16_ones();
  f32x4 acc[1][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int s0 = w; s0 < spans; s0 += D * kDecodeWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int span = s0 + d * kDecodeWaves;
      if (span >= spans) break;
      if constexpr (STAGED) {
        const int g = span * kSpan >> a.qw.lg_group;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          slot[d].sc[j].v[0] = steps[soff[j] + g];
          slot[d].zo[j].v[0] = zeros[soff[j] + g];
        }
      }
#pragma unroll
      for (int i = 0; i < PX; ++i) slot[d].xp[i].store(own[w], 4 * i + lq, lr);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      span_product<BITS, MODE, 1, NT>(own[w], slot[d].cw, slot[d].sc, slot[d].zo,
                                      a.K - span * kSpan < kSpan, mask, ones, lr, lq, acc);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (span + D * kDecodeWaves < spans) fetch(slot[d], span + D * kDecodeWaves);
    }
  }
  float* red = reinterpret_cast<float*>(own[w]);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(4 * lq + r) * LD + j * 16 + lr] = acc[0][j][r];
    } else {
      red[lq * LD + j * 16 + lr] = acc[0][j][0] + acc[0][j][1] + acc[0][j][2];
    }
  }
  if constexpr (LOCAL) nonzeros<RPW, true, false>(a, en, ent, k0, kend, beg, end, 1, zl, ad);
  __syncthreads();
  for (int e = threadIdx.x; e < toks * 16 * NT; e += kThreads) {
    const int t = e / (16 * NT), n = e % (16 * NT);
    if (n >= rows) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kDecodeWaves; ++i) v += __uint_as_float(own[i][t * LD + n]);
    if (!LOCAL && a.part != nullptr) {
      a.part[part_at(a, 0, t0 + t, n0 + n)] = v;
    } else {
      if constexpr (LOCAL) v = fmaf(a.alpha, ad[n][t], v);
      Elem<T>::st(y, static_cast<int64_t>(t0 + t) * a.N + n0 + n, v);
    }
  }
}

// ---- more tokens: 64 rows of tokens (64 bf16 or 16 fp32 ones) by 128 rows of W
// per workgroup, a wave 32 of them; the tokens' tiles are staged once for all
// waves, and the spans are split over `slices` workgroups, whose partial sums
// decode_finish_kernel adds up. Two spans are on their way while a third is
// worked on: with one the kernel waits for memory at every span. Of 27.6 us (8192 x
// 8192, 2 bits, 64 tokens; counters at 2.4 GHz) the vector instructions, most of
// them unpacking and the groups' steps, issue for 9.1 and the matrix cores are busy
// for 5.1; a SIMD's two waves wait for memory a third of their cycles, and the two
// kinds of work of one wave do not overlap. Deeper queues do not fit the 256
// registers: three spans on their way 34.0 -> 38.6 us, four 44.6 (8192 x 8192, 4
// bits, 64 tokens).
constexpr int kWideThreads = 256;
constexpr int kWideRows = 128;
constexpr int kWideTiles = 4;
constexpr int kWideGroups = 32;    // groups of a slice whose steps and zeros LDS holds

template <int BITS, int MODE, typename T>
__global__ __launch_bounds__(kWideThreads, 2) void decode_wide_kernel(const T* __restrict__ x,
                                                                      DecodeArgs a) {
  constexpr int MT = kWideTiles, NT = 2, G = 1 << MODE, D = 3;
  constexpr int TB = Rows<T>::TOK * MT;
  constexpr int PX = TB * 16 / kWideThreads;           // pieces of a span per thread
  using Code = Codes<BITS>;
  extern __shared__ __attribute__((aligned(16))) float dyn[];
  if (static_cast<int>(blockIdx.x) < a.z_blocks) {
    write_z<kWideThreads>(x, a, blockIdx.x, dyn);
    return;
  }
  uint32_t* tiles = reinterpret_cast<uint32_t*>(dyn);  // two buffers
  const int tiles_n = (a.N + kWideRows - 1) / kWideRows;
  int block = blockIdx.x - a.z_blocks;
  const int bn = block % tiles_n;
  block /= tiles_n;
  const int slice = block % a.slices, bt = block / a.slices;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int n0 = bn * kWideRows + w * 32, t0 = bt * TB;
  const int spans = (a.K + kSpan - 1) / kSpan;
  const int first = static_cast<int>(static_cast<int64_t>(spans) * slice / a.slices);
  const int last = static_cast<int>(static_cast<int64_t>(spans) * (slice + 1) / a.slices);

  // steps and zeros of the slice's groups for the workgroup's rows, in LDS
  const int g0 = first * kSpan >> a.qw.lg_group;
  const int ng = min((last * kSpan - 1 >> a.qw.lg_group) + 1, a.qw.gpr) - g0;
  float* steps = dyn + 2 * kWideTiles * kTileWords;
  float* zeros = steps + kWideRows * (kWideGroups + 1);
  const bool staged = ng <= kWideGroups;
  if (staged) {
    const int rows = min(kWideRows, a.N - bn * kWideRows);
    const float* s = a.qw.scales + static_cast<int64_t>(bn) * kWideRows * a.qw.gpr + g0;
    const float* z = a.qw.zeros + static_cast<int64_t>(bn) * kWideRows * a.qw.gpr + g0;
    const int g = tid & (kWideGroups - 1);
    if (g < ng) {
#pragma unroll 4
      for (int r = tid / kWideGroups; r < rows; r += kWideThreads / kWideGroups) {
        steps[r * (kWideGroups + 1) + g] = s[r * a.qw.gpr + g];
        zeros[r * (kWideGroups + 1) + g] = z[r * a.qw.gpr + g];
      }
    }
  }

  const int nb = min(n0, a.N - 1);                      // waves past N repeat the last row
  const uint32_t* ctile = a.qw.codes + static_cast<int64_t>(nb) * a.qw.wpr;
  const float* stile = a.qw.scales + static_cast<int64_t>(nb) * a.qw.gpr;
  const float* ztile = a.qw.zeros + static_cast<int64_t>(nb) * a.qw.gpr;
  uint32_t coff[NT], soff[NT], xoff[PX];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = min(j * 16 + lr, a.N - 1 - nb);
    coff[j] = 4u * n * a.qw.wpr;
    soff[j] = 4u * n * a.qw.gpr;
  }
  const int tok = tid >> 4, piece = tid & 15;
#pragma unroll
  for (int i = 0; i < PX; ++i)
    xoff[i] = sizeof(T) * min(t0 + 16 * i + tok, a.tokens - 1) * a.K;

  struct Slot {
    Code cw[NT];
    Groups<G> sc[NT], zo[NT];
    Piece<T> xp[PX];
  } slot[D];
  // Every workgroup starts at a span of its own. In step they would all read the
  // same columns, and rows a power of two apart meet in few of the L2's
  // channels.
  const int count = last - first, turn = (bn + slice) % max(count, 1);
  auto span_at = [&](int i) {
    const int r = i + turn;
    return first + (r < count ? r : r - count);
  };
  auto fetch = [&](Slot& s, int i) {
    const int span = span_at(i), c0 = span * kSpan;
#pragma unroll
    for (int i = 0; i < PX; ++i) s.xp[i].load(x, xoff[i], min(c0 + 8 * piece, a.K - 8));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      s.cw[j].load(ctile, coff[j], min(c0 + 32 * lq, a.K - 32));
      if (!staged) {
        s.sc[j].load(stile, soff[j], c0 >> a.qw.lg_group, a.qw.gpr);
        s.zo[j].load(ztile, soff[j], c0 >> a.qw.lg_group, a.qw.gpr);
      }
    }
  };
  const uint32_t mask = in_vgpr(Code::MASK);
  const bf16x8 ones = bf16_ones();
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (d < count) fetch(slot[d], d);
  int buf = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i0 + d >= count) break;
      // the buffer of the span before the last one: every wave is past the
      // barrier that follows its reads
      uint32_t* tb = tiles + buf * (MT * kTileWords);
      buf ^= 1;
#pragma unroll
      for (int i = 0; i < PX; ++i) {
        if constexpr (sizeof(T) == 2)
          slot[d].xp[i].store(tb + i * kTileWords, tok, piece);
        else
          slot[d].xp[i].store(tb + (tok >> 2) * kTileWords, tok & 3, piece);
      }
      if (i0 + d + D - 1 < count) fetch(slot[(d + D - 1) % D], i0 + d + D - 1);
      __syncthreads();
      if (staged) {
        const int g = (span_at(i0 + d) * kSpan >> a.qw.lg_group) - g0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int at = (w * 32 + j * 16 + lr) * (kWideGroups + 1);
#pragma unroll
          for (int k = 0; k < G; ++k) {
            slot[d].sc[j].v[k] = steps[at + min(g + k, ng - 1)];
            slot[d].zo[j].v[k] = zeros[at + min(g + k, ng - 1)];
          }
        }
      }
      span_product<BITS, MODE, MT, NT>(tb, slot[d].cw, slot[d].sc, slot[d].zo,
                                       a.K - span_at(i0 + d) * kSpan < kSpan, mask, ones, lr, lq,
                                       acc);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + j * 16 + lr;
      if (n >= a.N) continue;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = t0 + i * 16 + 4 * lq + r;
          if (t < a.tokens) a.part[part_at(a, slice, t, n)] = acc[i][j][r];
        }
      } else {
        const int t = t0 + i * 4 + lq;
        if (t < a.tokens)
          a.part[part_at(a, slice, t, n)] = acc[i][j][0] + acc[i][j][1] + acc[i][j][2];
      }
    }
}

// y = the slices' sums and the nonzeros of 8 RPW rows of F (SPLIT: of one), for up
// to 64 tokens. Bound by the gather of z's columns from L2 (64 tokens: 256 bytes a
// nonzero, 268 MB in 20 us) and, with few tokens, by the way from row_ptr over E
// to z: the partial sums are therefore fetched ahead of it.
template <typename T, int RPW, bool SPLIT>
__global__ __launch_bounds__(kThreads) void decode_finish_kernel(DecodeArgs a,
                                                                 T* __restrict__ y) {
  static_assert(!SPLIT || RPW == 1, "a row takes whole waves");
  constexpr int RB = SPLIT ? 1 : 8 * RPW;
  __shared__ float ad[8 * RPW][64 + 4];
  __shared__ uint2 ent[kEntries];
  constexpr int EACH = RB * 64 / kThreads > 1 ? RB * 64 / kThreads : 1;   // results of a thread
  constexpr int EARLY = 8;       // slices whose sums are fetched ahead of the nonzeros
  const int n0 = blockIdx.x * RB;
  const int64_t step = static_cast<int64_t>((a.N + 15) >> 4) * a.tokens * 16;
  const float* p[EACH];
  float q[EACH][EARLY];
  auto fetch = [&] {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int e = min(static_cast<int>(threadIdx.x) + i * kThreads, a.tokens * RB - 1);
      p[i] = a.part + part_at(a, 0, e / RB, min(n0 + e % RB, a.N - 1));
#pragma unroll
      for (int k = 0; k < EARLY; ++k)
        if (k < a.slices) q[i][k] = p[i][k * step];
    }
  };
  if (a.row_ptr != nullptr) {
    const int k0 = a.row_ptr[n0], kend = a.row_ptr[min(n0 + RB, a.N)];
    const int row = SPLIT ? n0 : n0 + threadIdx.x / (64 / RPW);
    const int beg = a.row_ptr[min(row, a.N)], end = a.row_ptr[min(row + 1, a.N)];
    fetch();
    Entries en;
    en.load(a, k0, kend);
    nonzeros<RPW, false, SPLIT>(a, en, ent, k0, kend, beg, end, a.tp / 4, nullptr, ad);
    __syncthreads();
  } else {
    fetch();
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = threadIdx.x + i * kThreads, t = e / RB, n = e % RB;
    if (e >= a.tokens * RB || n0 + n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < EARLY; ++k)
      if (k < a.slices) v += q[i][k];
#pragma unroll 4
    for (int k = EARLY; k < a.slices; ++k) v += p[i][k * step];
    if (a.row_ptr != nullptr) {
      float f = ad[n][t];
      if constexpr (SPLIT)
#pragma unroll
        for (int k = 1; k < kDecodeWaves; ++k) f += ad[k][t];
      v = fmaf(a.alpha, f, v);
    }
    Elem<T>::st(y, static_cast<int64_t>(t) * a.N + n0 + n, v);
  }
}

// ---- launches
template <typename T>
hipError_t finish(const DecodeArgs& a, T* y, hipStream_t s) {
  auto go = [&](auto kernel, int rows) {
    hipLaunchKernelGGL(kernel, dim3((a.N + rows - 1) / rows), dim3(kThreads), 0, s, a, y);
    return hipGetLastError();
  };
  // Rows per workgroup by what keeps the chip busy: one where there are few rows
  // or they are longer than that (8192 columns, T = 4, whole call with one / 8 rows:
  // 256 rows of 512 nonzeros 12.1 / 15.9 us, 1024 rows of 128, 512 and 1024
  // 14.9 / 12.5, 16.4 / 16.4 and 18.4 / 20.7, 4096 rows of 1024 44 / 34), 8
  // up to two workgroups per compute unit, 16 beyond (4096 columns, T = 16, 128
  // nonzeros a row, whole call with 8 / 16 / 32 rows: 4096 rows 19.0 / 19.4 / 24.9
  // us, 5120 rows 23.3 / 21.1 / 25.6, 14336 rows 38.4 / 33.7 / 35.7).
  if (a.row_ptr != nullptr && (a.N <= 512 || a.p / a.N > a.N - a.N / 4))
    return go(decode_finish_kernel<T, 1, true>, 1);
  if (a.N <= 4096) return go(decode_finish_kernel<T, 1, false>, 8);
  return go(decode_finish_kernel<T, 2, false>, 16);
}

size_t z_lds(const DecodeArgs& a) {
  return a.z_blocks > 0 ? static_cast<size_t>(a.z_cols + a.z_cols / 16) * 4 : 0;
}

template <typename T>
int token_tiles(int tokens) { return (tokens + Rows<T>::TOK - 1) / Rows<T>::TOK; }

template <int BITS, int MODE, int NT, typename T, bool FEW, bool LOCAL>
hipError_t decode_t(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  const size_t staged = MODE == kWide ? static_cast<size_t>(32) * NT * (a.qw.gpr + 1) * 4 : 0;
  const size_t local = LOCAL ? static_cast<size_t>(a.tokens) * (a.K + a.K / 16) * 4 : 0;
  const size_t lds = staged + local > z_lds(a) ? staged + local : z_lds(a);
  hipLaunchKernelGGL((decode_kernel<BITS, MODE, NT, T, FEW, LOCAL>),
                     dim3(a.z_blocks + (a.N + 16 * NT - 1) / (16 * NT) * token_tiles<T>(a.tokens)),
                     dim3(kThreads), lds, s, x, a, y);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && a.part != nullptr ? finish(a, y, s) : e;
}

constexpr int kUnits = 256, kLds = 163840;    // compute units; LDS of one

// Tiles of 16 rows a workgroup of decode_kernel takes: two where one would need
// more workgroups than there are compute units. The compute units that get a
// second one set the time (4096 columns, 16 tokens with one / two: 3584 rows 14.1 /
// 15.8 us, 4000 rows 18.1 / 15.9, 28672 rows 54 / 45; one token, LOCAL, 8192 rows
// 16.9 / 12.2). `others`: workgroups that transform tokens of 5 or more, whole
// ones of 4096 columns; smaller ones, and those beside the lighter tiles of few
// tokens, are over before it counts (4096 x 14336, 3 tokens 21.2 / 25.1, 8 tokens
// 22.4 / 23.7).
int row_tiles(int others, int N) { return others + (N + 15) / 16 > kUnits ? 2 : 1; }

// Whether every workgroup transforms the tokens for itself. That saves a launch
// and z's way through memory and costs each workgroup the transform, so: one
// token, or several of few columns (4096 rows, 128 nonzeros a row, us with the
// transform in LDS / through memory: 1 x 4096 9.7 / 11.1, 4 x 1024 8.9 / 9.3, 4 x
// 4096 13.8 / 11.9); nonzeros that one round of entries holds (1 x 2048: 64 a row
// 7.4 / 8.8, 256 11.2 / 11.1, 512 x 4 tokens 24.4 / 15.3); and all workgroups at
// once, or two at a time on a compute unit (1 x 4096: 8192 rows 11.9 / 14.3, 9216
// rows 21.1 / 19.5; 1 x 2048: 9216 rows 13.7 / 16.9).
bool is_local(int T, int K, int N, int64_t p) {
  if (p == 0 || T > kLocalTokens || T * K > (T == 1 ? kLocalOne : kLocal)) return false;
  const int nt = row_tiles(0, N);
  const int blocks = (N + 16 * nt - 1) / (16 * nt);
  const int lds = 65536 + nt * (512 + K + 128) + T * (K + K / 16) * 4;   // steps: groups of 128
  return 16 * nt * T * (p / N) <= kEntries && (blocks <= kUnits ? lds <= kLds : 2 * lds <= kLds);
}

// Whether decode_wide_kernel takes the product: where decode_kernel, a workgroup
// for every tile of tokens and two tiles of rows, and those that write z are more
// than the compute units (17 tokens of 4096 columns without an adapter, us with
// decode_kernel / decode_wide_kernel: 64 rows 6.0 / 8.5, 1024 rows 6.3 / 9.8, 4096
// rows 9.4 / 15.4, 8192 rows 17.6 / 17.9, 14336 rows 31.9 / 23.2; with 64 nonzeros
// a row and 40 tokens: 1024 rows 15.3 / 18.2, 2720 rows of 1024 columns 16.6 / 15.1,
// 64 rows of 14336 columns 21.0 / 16.7).
template <typename T>
bool is_wide(int tokens, int N, int z_blocks) {
  const int tiles = token_tiles<T>(tokens);
  return tiles > 1 && tiles * ((N + 31) / 32) + z_blocks > kUnits;
}

template <int BITS, int MODE, typename T>
hipError_t decode_m(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  if (is_wide<T>(a.tokens, a.N, a.z_blocks)) {
    constexpr int TB = Rows<T>::TOK * kWideTiles;
    const int blocks = (a.N + kWideRows - 1) / kWideRows * ((a.tokens + TB - 1) / TB) * a.slices;
    const size_t tiles = sizeof(uint32_t) * 2 * kWideTiles * kTileWords +
                         sizeof(float) * 2 * kWideRows * (kWideGroups + 1);
    hipLaunchKernelGGL((decode_wide_kernel<BITS, MODE, T>), dim3(a.z_blocks + blocks),
                       dim3(kWideThreads), tiles > z_lds(a) ? tiles : z_lds(a), s, x, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? finish(a, y, s) : e;
  }
  if (a.tokens <= 4) {
    if (is_local(a.tokens, a.K, a.N, a.p))
      return row_tiles(0, a.N) == 2 ? decode_t<BITS, MODE, 2, T, true, true>(x, a, y, s)
                                    : decode_t<BITS, MODE, 1, T, true, true>(x, a, y, s);
    return row_tiles(0, a.N) == 2 ? decode_t<BITS, MODE, 2, T, true, false>(x, a, y, s)
                                  : decode_t<BITS, MODE, 1, T, true, false>(x, a, y, s);
  }
  constexpr bool FEW = sizeof(T) == 4;       // tiles of 4 fp32 tokens
  return row_tiles(a.log_b >= 12 ? a.z_blocks : 0, a.N * token_tiles<T>(a.tokens)) == 2
             ? decode_t<BITS, MODE, 2, T, FEW, false>(x, a, y, s)
             : decode_t<BITS, MODE, 1, T, FEW, false>(x, a, y, s);
}

template <int BITS, typename T>
hipError_t decode_b(const T* x, const DecodeArgs& a, T* y, hipStream_t s) {
  if (a.qw.lg_group == 5) return decode_m<BITS, kFull, T>(x, a, y, s);
  if (a.qw.lg_group == 6) return decode_m<BITS, kHalf, T>(x, a, y, s);
  return decode_m<BITS, kWide, T>(x, a, y, s);
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

// tokens a column of zt holds: a power of two, 4 at least
int padded_tokens(int T) {
  int tp = 4;
  while (tp < T) tp *= 2;
  return tp;
}

// Workgroups that share the spans of 128 rows: with one a token that writes z two
// per compute unit, which is what fits at once; at least two spans each. Widths
// that are not a power of two may have several workgroups a token for z: some of
// the launch then wait for a second turn (4096 x 14336, 64 tokens: 448 of each
// kind for 512 places, 52.2 us; 11008 columns 45.1).
int wide_slices(int z_tokens, int K, int N) {
  const int tiles = (N + kWideRows - 1) / kWideRows, spans = (K + kSpan - 1) / kSpan;
  const int want = (512 - z_tokens) / tiles, most = spans / 2;
  const int n = want < most ? want : most;
  return n < 1 ? 1 : n;
}

struct DecodeWs {
  size_t part, total;     // zt at 0
};
// Calls of both types find room: fp32 ones may take decode_wide_kernel from 5
// tokens on, bf16 ones from 17.
DecodeWs decode_ws(int T, int K, int N, int64_t p) {
  DecodeWs l;
  const bool z = p > 0 && !is_local(T, K, N, p);
  l.part = z ? static_cast<size_t>(K) * padded_tokens(T) * 4 : 0;
  const size_t sums = static_cast<size_t>(T) * ((N + 15) / 16 * 16) * 4;
  l.total = l.part + (T > Rows<float>::TOK ? wide_slices(z ? T : 0, K, N) * sums : z ? sums : 0);
  return l;
}

}  // namespace

size_t decode_scratch_bytes(int T, int K, int N, int64_t p) { return decode_ws(T, K, N, p).total; }

hipError_t launch_decode(const void* x, Dt dt, int T, int log_n, int nblk, int N,
                         const QuantW& qw, int64_t p, const int32_t* row_ptr, const int32_t* E,
                         const float* c, float alpha, void* y, void* scratch, hipStream_t s) {
  DecodeArgs a;
  a.tokens = T;
  a.K = nblk << log_n;
  a.N = N;
  a.tp = padded_tokens(T);
  a.qw = qw;
  a.row_ptr = p > 0 ? row_ptr : nullptr;
  a.E = E;
  a.c = c;
  a.log_b = log_n;
  const bool through_memory = p > 0 && !is_local(T, a.K, N, p);
  a.p = p;
  // whole blocks of columns, 2048 together at least, in one workgroup
  a.z_cols = log_n >= 11 ? 1 << log_n : 2048;
  a.z_blocks = through_memory ? T * ((a.K + a.z_cols - 1) / a.z_cols) : 0;
  const bool wide = dt == Dt::F32 ? is_wide<float>(T, N, a.z_blocks)
                                  : is_wide<uint16_t>(T, N, a.z_blocks);
  a.part = wide || through_memory
               ? reinterpret_cast<float*>(static_cast<char*>(scratch) + decode_ws(T, a.K, N, p).part)
               : nullptr;
  a.slices = wide ? wide_slices(through_memory ? T : 0, a.K, N) : 1;
  a.z_out = static_cast<float*>(scratch);
  a.zt = a.z_out;
  a.alpha = through_memory ? alpha : alpha / static_cast<float>(1 << log_n);
  if (dt == Dt::F32) return decode_d(static_cast<const float*>(x), a, static_cast<float*>(y), s);
  return decode_d(static_cast<const uint16_t*>(x), a, static_cast<uint16_t*>(y), s);
}

}  // namespace qwha
