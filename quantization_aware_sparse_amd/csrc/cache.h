// The paged key/value cache as the kernels see it.
#pragma once

#include <type_traits>

#include "common.h"
#include "launch.h"

namespace qwha {

// codes [2][n_pages][heads][page][words], scales and zeros
// [2][n_pages][heads][page]: keys (part 0), then values. A head's tokens of a
// page lie together, so that attention reads a head's rows in whole lines.
struct Cache {
  uint32_t* codes;
  float* scales;
  float* zeros;
  int64_t n_pages;
  int lg_page;
  int heads;
  int dim, bits;
  // x / heads = (x * heads_magic) >> heads_shift for x < 2^31, with
  // 2^(shift - 31) the next power of two from heads on and magic =
  // ceil(2^shift / heads): x (magic heads - 2^shift) < 2^31 heads <= 2^shift
  uint32_t heads_magic;
  int heads_shift;

  __host__ __device__ uint32_t over_heads(uint32_t x) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(x) * heads_magic) >> heads_shift);
  }
  // rows of one part; the offsets of a long cache pass 32 bits
  __host__ __device__ int64_t part_rows() const { return (n_pages * heads) << lg_page; }
  // part * n_pages + page fits 32 bits (n_pages < 2^28): one 64-bit product
  __host__ __device__ int64_t row_in(int part, int32_t page, int off, int head) const {
    const uint32_t g = static_cast<uint32_t>(part) * static_cast<uint32_t>(n_pages) +
                       static_cast<uint32_t>(page);
    return static_cast<int64_t>(((static_cast<uint64_t>(g) * static_cast<uint32_t>(heads) +
                                  static_cast<uint32_t>(head)) << lg_page) +
                                static_cast<uint32_t>(off));
  }
  __host__ __device__ int64_t row(int part, int32_t slot, int head) const {
    return row_in(part, slot >> lg_page, slot & ((1 << lg_page) - 1), head);
  }
};

inline Cache make_cache(uint32_t* codes, float* scales, float* zeros, int64_t n_pages, int lg_page,
                        int heads, int dim, int bits) {
  int s = 0;
  while ((1 << s) < heads) ++s;
  const uint64_t one = uint64_t{1} << (31 + s);
  return Cache{codes, scales, zeros, n_pages, lg_page, heads, dim, bits,
               static_cast<uint32_t>((one + heads - 1) / heads), 31 + s};
}

// Calls fn with the kernel's compile-time choices.
template <typename Fn>
hipError_t by_shape(int dim, int bits, Fn&& fn) {
  using std::integral_constant;
  if (bits == 4) {
    if (dim == 64) return fn(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (dim == 128) return fn(integral_constant<int, 128>{}, integral_constant<int, 4>{});
    if (dim == 256) return fn(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  } else if (bits == 8) {
    if (dim == 64) return fn(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    if (dim == 128) return fn(integral_constant<int, 128>{}, integral_constant<int, 8>{});
    if (dim == 256) return fn(integral_constant<int, 256>{}, integral_constant<int, 8>{});
  }
  return hipErrorInvalidValue;
}

// q_heads / heads query heads read each head; max_tokens = width * page
size_t cache_attn_scratch_bytes(int B, int q_heads, int heads, int dim, int64_t max_tokens,
                                int page);
// workgroups along the first dimension of a launch's grid, which holds 2^32 - 1 threads
int64_t cache_attn_blocks(int B, int q_heads, int heads, int dim, int64_t max_tokens, int page);
constexpr int64_t kMaxAttnBlocks = 0xFFFFFFFFll / 256;
constexpr float kLog2E = 1.44269504088896340736f;
constexpr int kWritePer = 32;      // columns a lane of the writing kernel
constexpr int64_t kMaxWriteThreads = 0xFFFFFFFFll - 255;
hipError_t launch_cache_write(const void* k, const void* v, Dt dt, int64_t T,
                              const int32_t* slots, int rotate, const Cache& c, hipStream_t s);
hipError_t launch_cache_read(const Cache& c, const int32_t* slots, int64_t T, int rotate, Dt dt,
                             void* k, void* v, hipStream_t s);
hipError_t launch_cache_attn(const void* q, Dt dt, int B, int q_heads, const Cache& c,
                             const int32_t* table, int width, const int32_t* lens, float scale,
                             int rotate, void* out, void* scratch, hipStream_t s);

}  // namespace qwha
