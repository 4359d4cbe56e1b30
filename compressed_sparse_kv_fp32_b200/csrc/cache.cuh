// The cache geometry shared by the cache operators: where the rows of one token of
// one (b, kv head) live, in a contiguous cache or behind a block table.
#pragma once

#include "common.cuh"

namespace adamas {

constexpr uint32_t kErrOffsets = 0x10u;  // mirrors ADAMAS_DEVERR_OFFSETS in adamas.h

// n / d for any n < 2^31 by one multiplication (round-up reciprocal of d with
// s = ceil(log2 d): the error term n (2^s - ...) / 2^(32 + s) stays below 1 / d).
struct FastDiv {
  uint32_t d = 1, mul = 0, shift = 0;
  __host__ static FastDiv of(uint32_t d) {
    FastDiv f;
    f.d = d;
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    f.shift = s;
    f.mul = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};

struct CacheGeom {
  const int32_t* table;  // null: contiguous
  int64_t Nmax;          // tokens of a sequence (paged: max_pages * page_size)
  int64_t n_pages;
  int max_pages;
  int Hkv;
  FastDiv page;

  // Row of token t (0 <= t < Nmax) of (b, h).  A table entry outside [0, n_pages)
  // gives page 0 and sets bad.
  __device__ __forceinline__ int64_t row(int b, int h, int t, bool& bad) const {
    if (table == nullptr) return ((int64_t)b * Hkv + h) * Nmax + t;
    const uint32_t pg = page.div((uint32_t)t);
    const int slot = t - (int)(pg * page.d);
    int64_t phys = table[(int64_t)b * max_pages + pg];
    const bool out = phys < 0 || phys >= n_pages;
    bad |= out;
    phys = out ? 0 : phys;
    return (phys * Hkv + h) * page.d + slot;
  }
  // The same in 32 bits, for caches of rows that real memory holds (2^32 rows are a
  // terabyte).
  __device__ __forceinline__ uint32_t row32(int b, int h, int t, bool& bad) const {
    if (table == nullptr) return (uint32_t)(b * Hkv + h) * (uint32_t)Nmax + (uint32_t)t;
    const uint32_t pg = page.div((uint32_t)t);
    const uint32_t slot = (uint32_t)t - pg * page.d;
    uint32_t phys = (uint32_t)table[(int64_t)b * max_pages + pg];
    const bool out = phys >= (uint64_t)n_pages;  // a negative entry is a large one
    bad |= out;
    phys = out ? 0u : phys;
    return (phys * (uint32_t)Hkv + (uint32_t)h) * page.d + slot;
  }
};

__device__ __forceinline__ int64_t clamp_len(int64_t len, int64_t Nmax, bool& bad) {
  if (len < 0 || len > Nmax) {
    bad = true;
    return len < 0 ? 0 : Nmax;
  }
  return len;
}

// The rows [first, first + n) of sequence b in a packed batch of T rows.  Offsets that
// are not ascending within [0, T] give n = 0 and set bad.
__device__ __forceinline__ void ragged_rows(const int32_t* cu, int b, int T, int& first, int& n, bool& bad) {
  const int a = cu[b], e = cu[b + 1];
  const bool out = a < 0 || e < a || e > T;
  bad |= out;
  first = out ? 0 : a;
  n = out ? 0 : e - a;
}

}  // namespace adamas
