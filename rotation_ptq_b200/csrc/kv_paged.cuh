// The paged KV cache as the kernels see it, and the ragged batch that
// addresses it.
#pragma once

#include <stdint.h>

#include "../../include/sq.h"

namespace sq {
namespace paged {

constexpr int D = 128;

// Pages are head-major: codes [pages][hkv][page][D * bits / 8], scale and
// zero [pages][hkv][page].  Consecutive tokens of one head are contiguous
// inside a page, so attention reads a head's rows, scales and zero points in
// long runs (token-major rows would put them hkv rows apart and fetch every
// head's scales with each head's).
struct Pages {
  uint8_t* kc;
  float* ks;
  uint8_t* kz;
  uint8_t* vc;
  float* vs;
  uint8_t* vz;
  int64_t num_pages;
  int lps;       // log2(page size)
  int hkv;
};

// New tokens of B sequences, packed: sequence b's are rows cu[b] .. cu[b+1]-1.
struct Batch {
  const int32_t* table;   // [B][width] page numbers
  const int32_t* cu;      // [B + 1]
  const int32_t* len;     // [B]: tokens in the cache (before or with the new ones, by call)
  int width, B;
  int64_t T;
};

// Group index (row of the scale arrays) of (page, head, row in page).
__device__ __forceinline__ int64_t group_of(const Pages& P, int page, int head, int row) {
  return ((static_cast<int64_t>(page) * P.hkv + head) << P.lps) + row;
}

// The sequence that packed token t belongs to and its cache position, from
// cached lengths `len`.  Returns false for a token behind the last sequence
// (silently) or one whose lengths or page make no sense (bad = true).
__device__ __forceinline__ bool locate(const Pages& P, const Batch& b, int64_t t, int& pos,
                                       int& page, bool& bad) {
  bad = false;
  if (t >= b.cu[b.B] || t < b.cu[0]) return false;
  int lo = 0, hi = b.B;                    // cu[lo] <= t < cu[hi] when cu does not decrease
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t nth = t - b.cu[lo];
  const int64_t p = nth + b.len[lo];
  bad = true;
  if (b.len[lo] < 0 || nth < 0 || t >= b.cu[lo + 1] || p >= (static_cast<int64_t>(b.width) << P.lps))
    return false;
  page = b.table[static_cast<int64_t>(lo) * b.width + (p >> P.lps)];
  if (page < 0 || page >= P.num_pages) return false;
  pos = static_cast<int>(p);
  bad = false;
  return true;
}

}  // namespace paged
}  // namespace sq
