// Index arithmetic of the paged-cache kernels, the same on the host (which
// prepares it, and tests it through the debug build) and on the device.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#define QSA_HD __host__ __device__ __forceinline__

namespace qsa {

// x / y for 0 <= x, 0 < y: in 32 bits where both fit (a 64-bit division is a
// routine of about a hundred instructions).
QSA_HD int64_t div64(int64_t x, int64_t y) {
  if (((uint64_t)(x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

// j / page_size for 0 <= j < 2^31 by a multiplication (round-up method of
// Granlund and Montgomery): shift s with 2^s >= page_size, multiplier
// floor(2^32 (2^s - page_size) / page_size) + 1.
struct PageDivision { uint32_t mul, shift; };
inline PageDivision page_division(int32_t page_size) {
  uint32_t s = 0;
  while (((int64_t)1 << s) < page_size) ++s;
  return {(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - (uint64_t)page_size)) / (uint64_t)page_size + 1), s};
}
QSA_HD uint32_t page_quotient(uint32_t mul, uint32_t shift, uint32_t j) {
#ifdef __CUDA_ARCH__
  const uint32_t high = __umulhi(mul, j);
#else
  const uint32_t high = (uint32_t)(((uint64_t)mul * j) >> 32);
#endif
  return (high + j) >> shift;
}

// `total` units laid end to end, cut evenly over `parts` CTAs: CTA c has the
// units [begin(c), begin(c + 1)), base of them or one more.
struct EvenCut {
  int64_t base, more;
  QSA_HD EvenCut(int64_t total, int64_t parts) : base(div64(total, parts)), more(total - base * parts) {}
  QSA_HD int64_t begin(int64_t c) const { return c * base + (c < more ? c : more); }
  // the CTA that has unit u < total
  QSA_HD int64_t owner(int64_t u) const {
    const int64_t longer = more * (base + 1);
    return u < longer ? div64(u, base + 1) : more + div64(u - longer, base);
  }
};

// The prefill's grid: the first tile slot of sequence `seq`, whose tokens start
// at `row` (rows outside 0 .. T count as the nearer end), with `per` query rows a
// token and `rows` of them to a tile.  At least as many slots lie before the next
// sequence's first as the sequence has tiles.  T per < 2^30.
QSA_HD int first_tile_slot(int seq, int row, int T, uint32_t per, uint32_t rows) {
  row = row < 0 ? 0 : row;
  row = row < T ? row : T;
  return (int)((uint32_t)row * per / rows) + seq;
}

}  // namespace qsa
