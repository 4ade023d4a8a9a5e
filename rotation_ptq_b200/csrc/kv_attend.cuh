// What the paged attention kernels share: parameters, the shape of a
// sequence's work, and the score rule.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kv_paged.cuh"
#include "sq_device.cuh"

namespace sq {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// From scores of 2^22 (log2 units: float32 steps of a half) on, the exponential's argument is rounded like the
// maximum's, in two steps: a fused multiply-add would tell them apart by more than weights have room for.
constexpr float kPlain = 4194304.0f;
constexpr int TILE = 128;                  // keys per CTA step of the streaming kernel

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t sq;                              // elements between tokens of q
  Pages pages;
  Batch batch;                             // len: tokens in the cache, the new ones included
  const int32_t* prefix_table;             // shared pages in front of every sequence, or null
  int prefix_len;
  int hq, G;                               // query heads, and per KV head
  float scale, cap;                        // cap 0: none
  int window;                              // 0: none
  const float* slopes;                     // [hq], or null
  __nv_bfloat16* out;                      // [T][hq][128]
  float* lse;                              // [T][hq], or null
  uint32_t spin_limit;
  // the streaming kernel: sequences of up to many_rows rows (others are the tile kernel's)
  int many_rows;
  unsigned* count;                         // workspace, zero at rest: one counter per CTA
  float* part;                             // null: units are not split
  // the tile kernel: sequences of more than few_rows rows, or all rows over the prefix (shared)
  int few_rows, shared, nsplit;
  int64_t units;
  unsigned* tcount;                        // workspace, zero at rest: one counter per unit
  float* tpart;                            // [units / nsplit][nsplit]: O [256][128], (m, l) [256]
  // the shared prefix's partial results, for the streaming kernel to join
  int ex_n;                                // pieces, 0: none
  float* ex_o;                             // [piece][T][hq][128]
  float* ex_ml;                            // [piece][T][hq][2]
  float inv_cap;                           // 1 / cap, at most 3e38: in the queries' factors a large cap leaves float32
};

// One sequence's new tokens and keys.  Positions count the shared prefix
// first: new token i sits at prefix_len + len - qlen + i, own cache row j at
// prefix_len + j.
struct Seq {
  int row0, qlen, len;                     // first packed row; new tokens; own cached tokens
  int pos0;                                // position of the first new token (may be negative)
  int pt0, pn, ot0, on;                    // first tile and tile count: prefix, own
  bool keys;                               // its lengths make sense
  __device__ __forceinline__ int tiles() const { return pn + on; }
};

// Reads sequence b; lengths that make no sense are reported and leave it
// without tokens (row range outside the batch) or without keys.
__device__ __forceinline__ Seq load_seq(const AttnParams& P, int b, bool report) {
  Seq s;
  s.row0 = P.batch.cu[b];
  const int end = P.batch.cu[b + 1];
  s.len = P.batch.len[b];
  s.qlen = end - s.row0;
  bool keys = true;
  if (s.row0 < 0 || end < s.row0 || end > P.batch.T) {
    s.row0 = s.qlen = 0;
    keys = false;
  }
  if (s.len < 0 || s.len > (static_cast<int64_t>(P.batch.width) << P.pages.lps)) keys = false;
  if (!keys) {
    if (report) record_status(SQ_ERR_INVALID_ARG);
    s.len = 0;
  }
  s.keys = keys;
  s.pos0 = P.prefix_len + s.len - s.qlen;
  int low = 0;                             // lowest visible position of any new token
  if (P.window > 0 && s.pos0 - P.window + 1 > 0) low = s.pos0 - P.window + 1;
  const int own_low = low > P.prefix_len ? low - P.prefix_len : 0;
  s.pt0 = low / TILE;
  s.pn = keys && s.qlen > 0 && low < P.prefix_len && P.ex_n == 0
             ? (P.prefix_len - 1) / TILE - s.pt0 + 1
             : 0;
  s.ot0 = own_low / TILE;
  s.on = keys && s.qlen > 0 && own_low < s.len ? (s.len - 1) / TILE - s.ot0 + 1 : 0;
  return s;
}

// tanh to about 1e-7 absolute; relative for small |x| (odd Taylor terms).
__device__ __forceinline__ float tanh_score(float x) {
  const float e = exp2f(2.0f * kLog2e * x);
  const float big = 1.0f - __fdividef(2.0f, e + 1.0f);
  const float y = x * x;
  const float small =
      x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 0.021869489f, -0.053968254f), 0.13333334f), -0.33333334f), 1.0f);
  return fabsf(x) < 0.25f ? small : big;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Four fp16 pairs (nibble i, nibble i + 4), i = 0..3, of a word of 8 codes,
// less the zero points z (lo half: the pair's first, hi half: its second).
// 0x6400 | n is 1024 + n, and 0x6400 | 16 n is 1024 + 16 n: one fma by 1/16
// takes the place of a shift.  All steps are exact.
__device__ __forceinline__ void widen_nibbles(uint32_t w, __half2 z1, __half2 z16, uint32_t (&o)[4]) {
  const __half2 sixteenth = __float2half2_rn(0.0625f);
  const uint32_t w8 = w >> 8;
  o[0] = h2_bits(__hadd2(bits_h2((w & 0x000F000Fu) | 0x64006400u), z1));
  o[1] = h2_bits(__hfma2(bits_h2((w & 0x00F000F0u) | 0x64006400u), sixteenth, z16));
  o[2] = h2_bits(__hadd2(bits_h2((w8 & 0x000F000Fu) | 0x64006400u), z1));
  o[3] = h2_bits(__hfma2(bits_h2((w8 & 0x00F000F0u) | 0x64006400u), sixteenth, z16));
}

// Two fp16 pairs (bytes 0, 1) and (2, 3) of a word of 4 codes, less z.
__device__ __forceinline__ void widen_bytes(uint32_t w, __half2 z1, uint32_t (&o)[2]) {
  o[0] = h2_bits(__hadd2(bits_h2(__byte_perm(w, 0x64646464u, 0x4140u)), z1));
  o[1] = h2_bits(__hadd2(bits_h2(__byte_perm(w, 0x64646464u, 0x4342u)), z1));
}

// What a call launches and the workspace it wants (kv_attend.cu).
struct AttnPlan {
  int kind;                                // streaming kernel: up to 4, 8 or 16 rows per unit
  bool stream, tile, shared;               // which kernels run; shared: the prefix pass
  int tile_split;                          // CTAs that may share a tile unit
  int64_t tile_units;
  size_t part, tpart, ex_o, ex_ml, bytes;  // offsets in the workspace, and its size
};

sq_status launch_tile(const AttnParams& P, int bits, cudaStream_t stream);

}  // namespace paged
}  // namespace sq
