// Attention of many rows over the paged 4/8-bit cache, sm_100a: the tile
// kernel on tcgen05.
//
// A unit is up to 256 rows (token, query head of one KV head) in two halves of
// 128, and a run of 128-key tiles.  Per half and tile
//     S = Q K_int^T            (tensor memory, f32; Q and codes exact in fp16)
//     y = S sk,  p = exp2(y f_row - m),  P = fp16(p sv)      (tensor memory)
//     O += P V_int             (A from tensor memory, f32)
// with K_int, V_int the codes less their zero points.  The row scales sk and
// sv stay outside the products, so fp16 operands lose nothing; P is rounded
// once to 11 bits, an eighth of what the bf16 output's own rounding may lose.
//
// Warps: 0-3 and 4-7 softmax of half 0 and 1, 8-11 widen codes from global
// memory into swizzled shared memory, 12 and 13 issue the halves' products, 14
// works out the units.  A step is 64 keys and each half has two buffers of
// scores, so that the next step's scores are there when a softmax ends; the
// halves run independently.
//
// What it took (prompts of 2 x 4096, 4 bits, us): an issuing warp whose
// descriptors do not spill, 920 to 710; the softmax's common case without
// branches, 566; one uniform issuing warp per half, 540 (a step's 12 products
// took 1500 cycles to issue from inside a branch, and 500 now); references with
// a slack, so that few steps rescale; the softmax in the fragment layout, where
// a lane needs the scales of a quarter of the keys (with a thread per row every
// lane reads them all: those broadcasts and the products' operand reads, both
// from shared memory, slow one another 1.5 times); caps and slopes compiled by
// themselves, 546 to 449 (the softmax's loop is a third shorter; more copies of
// its parts for special cases cost more than their branches: 510).  It is the
// code that counts, more than the times it runs: rows' own value scales in their
// references and scores of any size, all in a branch that few steps take, cost
// 449 to 477, and one copy of the issuing code for both halves instead of two
// gave 438 (445 with what caps of any size changed around it).  What bounds
// it is the softmax's own latency: when the whole took 541 us, it took 275
// without its arithmetic, 460 without the products, 446 without the widening and
// as long as before without the exponentials alone.
//
// Two kinds of work: a sequence's own rows over what it sees (splits of a
// unit's tiles are joined by the last CTA to arrive, in order), or, for a
// shared prefix, all sequences' rows over the prefix's tiles, whose partial
// results (O, m, l) the streaming kernel joins with each sequence's own part.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "kv_attend.cuh"
#include "sq_device.cuh"
#include "sq_host.h"

namespace sq {
namespace paged {

constexpr int KT = 128;                    // keys per tile
constexpr int HALF = 128;                  // rows per half
constexpr int TILE_THREADS = 16 * 32;      // warp 15 fills the last group
constexpr int UNITS = 3;                   // unit records in flight
constexpr int PANEL = 128 * 128;           // bytes of 128 rows x 64 fp16
constexpr int OFF_Q = 0;                   // [half][2 panels]
constexpr int OFF_K = OFF_Q + 4 * PANEL;   // [stage][2 panels]
constexpr int OFF_V = OFF_K + 4 * PANEL;
constexpr int OFF_SK = OFF_V + 4 * PANEL;  // float [4][KT]
constexpr int OFF_SV = OFF_SK + 4 * KT * 4;
constexpr int OFF_HID = OFF_SV + 4 * KT * 4;   // uint32 [4][8]: 4 words of hidden keys, 4 of flags
constexpr int OFF_SVE = OFF_HID + 128;         // float [4][4]: exponent above all value scales of 32 keys
constexpr int OFF_RUN = OFF_SVE + 64;          // uint8 [4][KT][8]: the same, biased, of the 2^k keys from one on
constexpr int OFF_BARS = OFF_RUN + 4 * KT * 8;
constexpr int OFF_UNITS = OFF_BARS + 512;      // TileUnit [UNITS]
constexpr int TILE_SMEM = OFF_UNITS + UNITS * 128 + 1024;
constexpr uint32_t TILE_TMEM = 512;        // S [half][64 keys], O [half]
constexpr uint32_t IDESC_S = idesc_f16(128, KT / 2, false, false);
// A row's reference is its largest score so far and the exponent of the largest value scale that it sees,
// less kTop (log2 units): weights (times the values' scales) reach 2^kTop and may pass it by kSlack more
// before the sums are rescaled (which costs as much as the rest of a step; with a slack of 1 it came in
// most of a prompt's steps).  fp16 then holds weights in full down to 2^-(14 + kTop) of the largest and in
// fixed steps of 2^-(24 + kTop) below.  A row's own scales count, since a hidden key's, however large, has
// no business with its weights' precision; where a step shows a row a part of its keys, the exponent
// is looked up by the run that it sees (prompts, when this came, 464 us, against 452 with one exponent for
// all of a warp's rows; 600 taken off the scores' registers, 530 in a loop over the keys).
constexpr float kTop = 10.0f, kSlack = 5.0f;
// Value scales are taken as they are while a step's largest is within 2^+-kEnds, else times a power of two,
// for all rows of the warp, that brings it to 2^+-kInside.  A row whose own are 2^-kReach and more of
// what they are then keeps its precision: beside hidden ones near float32's end, those from 2^-12 on.
constexpr float kEnds = 60.0f, kInside = 40.0f, kReach = 100.0f;
// The sums of exponentials are held at 2^-40 of themselves: beside large scales, exponentials are up to
// 2^(kTop + kSlack + kReach).
constexpr float kDown = 9.094947e-13f;
constexpr float kNone = -3.0e38f;          // the reference of a row that has seen no key
constexpr uint32_t IDESC_O = idesc_f16(128, 128, false, true);

struct TileBars {
  uint64_t k_full[2], v_full[2], k_free[2], v_free[2], sc_full[4];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2];        // [half][the tile's first or second 64 keys]
  uint64_t parts, joined, drain;           // partial results written; who joins them is known
  uint64_t u_full[UNITS], u_free[UNITS];
  uint32_t tmem, last;
};
static_assert(sizeof(TileBars) <= 512, "barriers");

// Products and commits under a predicate (the elected lane): the issuing warps' code stays uniform, so
// that descriptors are computed once for the warp and cost no moves (a branch around the products made
// a step of 12 take 1500 cycles to issue).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}

__device__ __forceinline__ void mma_f16_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void mma_f16_ts(uint32_t elected, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(elected)
      : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)), "r"(elected)
      : "memory");
}

// A unit as every role sees it.  Warp 14 works them out and hands them on in a ring of records in
// shared memory: the other roles hold only what they use.  rows 0: no unit follows.
struct TileUnit {
  int row0;                                // packed row of the first token
  int base, rows;                          // first (token, head) row of the unit, live rows
  int h, pos0;                             // KV head; position of token 0 (own rows)
  int len;                                 // own cached tokens
  const int32_t* table;                    // own pages
  int pt0, pn, ot0;                        // prefix tiles from pt0, pn of them, then own from ot0
  int first, n;                            // this CTA's tiles of the unit's list
  int steps;                               // of 64 keys: 2 n, or one less where the last sees nothing
  int pieces, piece;                       // how many CTAs share the unit; which one this is
  int slot;                                // the unit's place among the units
};

static_assert(sizeof(TileUnit) <= 128, "unit records");

// First tile of the shared prefix that some new token sees (by a warp).
__device__ __forceinline__ int first_shared_tile(const AttnParams& P) {
  if (P.window == 0) return 0;
  int least = 0x7fffffff;                  // position of the first new token of all
  for (int b = threadIdx.x & 31; b < P.batch.B; b += 32) {
    const Seq s = load_seq(P, b, false);
    if (s.keys && s.qlen > 0) least = min(least, s.pos0);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  return min(max(least - P.window + 1, 0), P.prefix_len - 1) / KT;
}

// Unit `x` of this launch; false if it is empty.  low_tile: first_shared_tile().
__device__ __forceinline__ bool tile_unit(const AttnParams& P, int64_t x, int low_tile, TileUnit& u) {
  const int G = P.G, hkv = P.pages.hkv, R = 2 * HALF;
  u.piece = static_cast<int>(x % P.nsplit);
  const int64_t y = x / P.nsplit;
  u.h = static_cast<int>(y % hkv);
  const int64_t z = y / hkv;
  u.slot = static_cast<int>(y);
  if (P.shared) {
    // all sequences' rows over the prefix
    const int64_t rows = static_cast<int64_t>(min(static_cast<int64_t>(P.batch.cu[P.batch.B]), P.batch.T)) * G;
    if (z * R >= rows) return false;
    u.row0 = 0;
    u.base = static_cast<int>(z) * R;
    u.rows = static_cast<int>(min(static_cast<int64_t>(R), rows - z * R));
    u.pos0 = 0;
    u.len = 0;
    u.table = nullptr;
    u.pt0 = low_tile;
    u.pn = (P.prefix_len - 1) / KT + 1 - low_tile;
    u.ot0 = 0;
    const int per = (u.pn + P.nsplit - 1) / P.nsplit;
    u.first = min(u.pn, u.piece * per);
    u.n = min(per, u.pn - u.first);
    u.steps = 2 * u.n;
    if (u.n > 0 && u.first + u.n == u.pn && ((P.prefix_len - 1) & (KT - 1)) < KT / 2) --u.steps;
    u.pieces = P.nsplit;
    return true;
  }
  // sequence b owns the places floor(cu[b] G / R) + b .. floor(cu[b + 1] G / R) + b, at least
  // as many as it has row blocks; the latest rows (which see most keys) come first
  const int32_t* cu = P.batch.cu;
  const int B = P.batch.B;
  auto place = [&](int b) { return static_cast<int64_t>(cu[b]) * G / R + b; };
  if (z >= place(B)) return false;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (place(mid) <= z)
      lo = mid;
    else
      hi = mid;
  }
  const Seq s = load_seq(P, lo, false);
  const int64_t rows = static_cast<int64_t>(s.qlen) * G;
  if (rows <= P.few_rows) return false;    // the streaming kernel's, which reports too
  const int blocks = static_cast<int>((rows + R - 1) / R);
  const int64_t back = place(lo + 1) - 1 - z;
  const int64_t rt64 = back - (place(lo + 1) - place(lo) - blocks);
  const int rt = rt64 >= 0 && rt64 < blocks ? static_cast<int>(rt64) : -1;
  if (rt < 0) return false;
  u.row0 = s.row0;
  u.base = rt * R;
  u.rows = static_cast<int>(min(static_cast<int64_t>(R), rows - u.base));
  u.pos0 = s.pos0;
  u.len = s.len;
  u.table = P.batch.table + static_cast<int64_t>(lo) * P.batch.width;
  const int p_first = s.pos0 + u.base / G, p_last = s.pos0 + (u.base + u.rows - 1) / G;
  const int low = P.window > 0 ? max(0, p_first - P.window + 1) : 0;
  const int high = s.keys ? min(p_last + 1, P.prefix_len + s.len) : 0;    // exclusive
  const int pre = min(high, P.prefix_len);
  u.pt0 = low / KT;
  u.pn = low < pre ? (pre - 1) / KT - u.pt0 + 1 : 0;
  const int own_low = max(0, low - P.prefix_len), own_high = high - P.prefix_len;
  u.ot0 = own_low / KT;
  const int total = u.pn + (own_low < own_high ? (own_high - 1) / KT - u.ot0 + 1 : 0);
  const int per = max((total + P.nsplit - 1) / P.nsplit, 2);     // two tiles a piece at least
  u.pieces = max(1, (total + per - 1) / per);
  if (u.piece >= u.pieces) return false;
  u.first = u.piece * per;
  u.n = min(per, total - u.first);
  u.steps = 2 * u.n;
  if (u.n > 0 && u.first + u.n == total &&
      ((total > u.pn ? own_high : pre) - 1) % KT < KT / 2)
    --u.steps;
  return true;
}

// Position of the first key of tile i of a unit.
__device__ __forceinline__ int tile_pos(const AttnParams& P, const volatile TileUnit& u, int i) {
  const int k = u.first + i, pn = u.pn;
  return k < pn ? (u.pt0 + k) * KT : P.prefix_len + (u.ot0 + k - pn) * KT;
}

// Tile i of a unit: its first row, row limit and position.
struct TileAt {
  const int32_t* table;
  int local, limit, kpos;
};
__device__ __forceinline__ TileAt tile_at(const AttnParams& P, const volatile TileUnit& u, int i) {
  const int k = u.first + i;
  if (k < u.pn) {
    const int l = (u.pt0 + k) * KT;
    return TileAt{P.prefix_table, l, P.prefix_len, l};
  }
  const int l = (u.ot0 + k - u.pn) * KT;
  return TileAt{u.table, l, u.len, P.prefix_len + l};
}

// The k-th unit of this CTA: rounds over the grid, every other one backwards,
// so that no CTA always gets a round's longest unit.
__device__ __forceinline__ int64_t unit_index(int k) {
  const int64_t g = gridDim.x;
  return k * g + ((k & 1) ? g - 1 - blockIdx.x : blockIdx.x);
}

// Where dim d of a group of 8 sits among the fp16 that a widened 4-bit word
// leaves: 0 4 1 5 2 6 3 7 from the front.
template <int BITS>
__device__ __forceinline__ constexpr int place8(int d) {
  return BITS == 8 ? d : (d < 4 ? 2 * d : 2 * (d - 4) + 1);
}

// Where 16-byte chunk c of a row of 256 bytes lies in two swizzled panels.
__device__ __forceinline__ int chunk_at(int row, int c) {
  return (c >> 3) * PANEL + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// Bits 0 .. n - 1, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Pairs of floats as the 64-bit registers that f32x2 instructions take: a pair that stays (a row's
// factor, twice) is put together once.
using pair_t = unsigned long long;
__device__ __forceinline__ pair_t pair_of(uint32_t x, uint32_t y) {
  pair_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(x), "r"(y));
  return p;
}
__device__ __forceinline__ pair_t pair_of(float x, float y) {
  return pair_of(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ float2 floats_of(pair_t p) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(p));
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ pair_t pair_mul(pair_t a, pair_t b) {
  pair_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ pair_t pair_add(pair_t a, pair_t b) {
  pair_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ pair_t pair_fma(pair_t a, pair_t b, pair_t c) {
  pair_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// (a, b) *= p, floats held in registers of tensor-memory transfers.
__device__ __forceinline__ void mul2u(uint32_t& a, uint32_t& b, pair_t p) {
  const float2 r = floats_of(pair_mul(pair_of(a, b), p));
  a = __float_as_uint(r.x);
  b = __float_as_uint(r.y);
}

// 2^e for a whole e of -126 .. 127.
__device__ __forceinline__ float power_of_two(float e) {
  return __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(e)) << 23);
}

// The largest of three; NaN loses, as with fmaxf.
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return y;
}

// Tensor memory in the fragment layout, 16 lanes (rows) at a time.  Lane (g, t) = (lane / 4, lane % 4)
// of the warp holds, of every group of 8 columns, columns 2t, 2t + 1 of row g (registers 4 i, 4 i + 1
// of group i) and of row g + 8 (4 i + 2, 4 i + 3); of 16-bit pairs, every group of 4 columns, column t
// of row g (2 i) and of row g + 8 (2 i + 1).
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256b_x1(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x256b_x1(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}


// ------------------------------------------------------------ widening

template <int BITS>
struct TileCodes {                         // a producer lane's share of one operand: 4 rows
  uint4 c[4][BITS / 4];
};

template <int BITS>
__device__ __forceinline__ void widen_rows(uint8_t* dst, const TileCodes<BITS>& v,
                                           int zeros, int warp_row, int rsub, int t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = warp_row + 8 * j + rsub;
    const uint32_t zero = __shfl_sync(0xffffffffu, zeros, 8 * j + rsub);  // of lane's row: warp_row + lane
    const __half2 z1 = bits_h2((zero * 0x00010001u) | 0xE400E400u);       // -(1024 + zero)
    uint8_t* line = dst + row * 128;
    if (BITS == 4) {
      const __half2 z16 = bits_h2((zero * 0x00100010u) | 0xD400D400u);    // -(64 + zero)
      const uint32_t w[4] = {v.c[j][0].x, v.c[j][0].y, v.c[j][0].z, v.c[j][0].w};
      const int odd = t >> 1;
#pragma unroll
      for (int e0 = 0; e0 < 4; ++e0) {
        // lanes of the second panel take their words in another order: no two of the eight
        // lanes of a store phase share a bank
        const uint32_t word = odd ? w[e0 ^ 1] : w[e0];
        const int chunk = (t & 1) * 4 + (e0 ^ odd);
        uint32_t o[4];
        widen_nibbles(word, z1, z16, o);
        *reinterpret_cast<uint4*>(line + odd * PANEL + ((chunk ^ (row & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < BITS / 4; ++q) {
        const uint32_t w[4] = {v.c[j][q].x, v.c[j][q].y, v.c[j][q].z, v.c[j][q].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a[2], b[2];
          widen_bytes(w[2 * e], z1, a);
          widen_bytes(w[2 * e + 1], z1, b);
          const int chunk = 2 * t + e;
          *reinterpret_cast<uint4*>(line + q * PANEL + ((chunk ^ (row & 7)) << 4)) =
              make_uint4(a[0], a[1], b[0], b[1]);
        }
      }
    }
  }
}

// The products of half H, by one warp.  Tensor memory is the whole SM's (512 columns), so its address is 0.
__device__ __forceinline__ void issue_products(int H, const AttnParams& P, uint8_t* smem, TileBars& bar,
                                               const TileUnit* ring_u) {
  const uint32_t t_s = H * 128, t_o = 256 + H * 128;
  const uint32_t spin = P.spin_limit, elected = elect_lane();
  bool ok = true;
  int tiles = 0;
  uint32_t par_q = 0, par_p = 0;           // parities that come next: q_full; bit b, p_full[b]
  const uint64_t q_desc = desc_sw128(smem_u32(smem + OFF_Q) + H * 2 * PANEL),
                 k_desc = desc_sw128(smem_u32(smem + OFF_K)),
                 v_desc = desc_sw128_mn(smem_u32(smem + OFF_V), PANEL, 1024);
  for (int k = 0, slot = 0, par_u = 0; ok; ++k) {
    ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_full[slot], par_u, spin));
    if (!ok) break;
    const volatile TileUnit& u = ring_u[slot];
    const int rows = __shfl_sync(0xffffffffu, u.rows, 0), n = __shfl_sync(0xffffffffu, u.n, 0),
              steps = __shfl_sync(0xffffffffu, u.steps, 0);
    if (rows == 0) break;
    __syncwarp();
    if (elected) mbar_arrive(&bar.u_free[slot]);
    if (++slot == UNITS) slot = 0, par_u ^= 1;
    if (H * HALF >= rows) {
      // a half without rows lets go of the tiles as they come
      for (int i = 0; i < n && ok; ++i) {
        const int tile = tiles + i;
        ok = mbar_wait(&bar.k_full[tile & 1], (tile >> 1) & 1, spin);
        if (ok && elected) mbar_arrive(&bar.k_free[tile & 1]);
        ok = ok && mbar_wait(&bar.v_full[tile & 1], (tile >> 1) & 1, spin);
        if (ok && elected) mbar_arrive(&bar.v_free[tile & 1]);
        ok = __all_sync(0xffffffffu, ok);
      }
      tiles += n;
      continue;
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&bar.q_full[H], par_q, spin));
    par_q ^= 1;
    // scores of step j, whose tile is there; they run two steps (the buffers) ahead of the products
    // with values
    auto scores = [&](int j) {
      const int stage = (tiles + (j >> 1)) & 1, b = j & 1;
      const uint64_t kd = k_desc + ((stage * 2 * PANEL + b * (PANEL / 2)) >> 4);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint32_t off = ((s >> 2) * PANEL + (s & 3) * 32) >> 4;
        mma_f16_ss(elected, t_s + b * (KT / 2), q_desc + off, kd + off, IDESC_S, s > 0);
      }
      commit_if(elected, &bar.s_full[H][b]);
      if (b || j == steps - 1) commit_if(elected, &bar.k_free[stage]);
    };
    if (ok && steps > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_full[tiles & 1], (tiles >> 1) & 1, spin));
      tc_fence_after();
      if (ok) {
        scores(0);
        if (steps > 1) scores(1);
      }
    }
    for (int j = 0; j < steps && ok; ++j) {
      const int tile = tiles + (j >> 1), stage = tile & 1, b = j & 1;
      ok = mbar_wait(&bar.p_full[H][b], (par_p >> b) & 1, spin);
      par_p ^= 1u << b;
      if (b == 0) ok = ok && mbar_wait(&bar.v_full[stage], (tile >> 1) & 1, spin);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = v_desc + ((stage * 2 * PANEL + b * (PANEL / 2)) >> 4);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_f16_ts(elected, t_o, t_s + b * (KT / 2) + 8 * s, vd + s * (2048 >> 4), IDESC_O, j > 0 || s > 0);
      commit_if(elected, &bar.o_full[H][b]);
      if (b || j == steps - 1) commit_if(elected, &bar.v_free[stage]);
      if (j + 2 < steps) {
        if (b == 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_full[stage ^ 1], ((tile + 1) >> 1) & 1, spin));
          if (!ok) break;
          tc_fence_after();
        }
        scores(j + 2);
      }
    }
    tiles += n;
  }
  // no product may still write the tensor memory freed when all have left
  commit_if(elected, &bar.drain);
  mbar_wait(&bar.drain, 0, 0);
  __syncwarp();
}

// SPECIAL: scores with a cap or slopes.  Without them the softmax is a third less code.
template <int BITS, bool SPECIAL>
__global__ void __launch_bounds__(TILE_THREADS, 1) tile_kernel(const AttnParams P) {
  constexpr int RB = D * BITS / 8;
  extern __shared__ uint8_t tile_smem_raw[];
  uint8_t* smem = tile_smem_raw + ((1024u - (smem_u32(tile_smem_raw) & 1023u)) & 1023u);
  float* s_sk = reinterpret_cast<float*>(smem + OFF_SK);
  float* s_sv = reinterpret_cast<float*>(smem + OFF_SV);
  uint32_t* s_hid = reinterpret_cast<uint32_t*>(smem + OFF_HID);
  float* s_sve = reinterpret_cast<float*>(smem + OFF_SVE);
  uint8_t* s_run = smem + OFF_RUN;
  TileBars& bar = *reinterpret_cast<TileBars*>(smem + OFF_BARS);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t spin = P.spin_limit;

  griddep_wait();                          // a programmatic dependent
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.k_free[i], 2);
      mbar_init(&bar.v_free[i], 2);
      mbar_init(&bar.q_full[i], 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bar.s_full[i][b], 1);
        mbar_init(&bar.p_full[i][b], 4);
        mbar_init(&bar.o_full[i][b], 1);
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bar.sc_full[i], 4);
    mbar_init(&bar.parts, 8);
    mbar_init(&bar.joined, 1);
    mbar_init(&bar.drain, 2);
    for (int i = 0; i < UNITS; ++i) {
      mbar_init(&bar.u_full[i], 1);
      mbar_init(&bar.u_free[i], 14);
    }
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&bar.tmem, TILE_TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  // What follows may be set up from here on: not before this kernel has its tensor memory, which a
  // follower that waits for this kernel's end might else hold.  Behind a shared prefix's pass it is the
  // streaming kernel that joins; it relies on the wait above for the call's inputs.
  griddep_launch_dependents();
  TileUnit* ring_u = reinterpret_cast<TileUnit*>(smem + OFF_UNITS);
  bool ok = true;

  // registers, of the 512 x 128 that the block is launched with: 128 x (2 x 192 + 64 + 64) at 4 bits,
  // 128 x (2 x 184 + 88 + 56) at 8
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(BITS == 4 ? 192 : 184));
    const int hf = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t t_s0 = lane_base + hf * 128, t_o = lane_base + 256 + hf * 128;
    const int r = 32 * quarter + lane;     // row within the half (a thread per row before and after the tiles)
    const int g = lane >> 2, t = lane & 3;
    int tiles = 0, splits = 0;             // tiles seen by the CTA; joins
    uint32_t par_s = 0, par_o = 0;         // bit b: parities that come next, s_full[b] and o_full[b]
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_full[k % UNITS], (k / UNITS) & 1, spin));
      if (!ok) break;
      const volatile TileUnit& u = ring_u[k % UNITS];
      const int rows = u.rows, n = u.n, steps = u.steps;
      if (rows == 0) break;
      const bool active = hf * HALF < rows;
      const int row = hf * HALF + r;
      // the rows of this thread's fragments: 16 bk + 8 i + g at index 2 bk + i
      float m[4] = {kNone, kNone, kNone, kNone}, l[4] = {0.f, 0.f, 0.f, 0.f};
      float sv_exp = -1000.f;                // value scales are taken times 2^-sv_exp; the first step sets it
      bool far = false;                      // it is not 0, or a row's scores are past kPlain
      if (active) {
        const int at = u.base + min(row, rows - 1), tok = at / P.G, head = u.h * P.G + at - tok * P.G;
        int row_pos = u.pos0 + tok;
        if (P.shared) {
          // the packed token's own sequence
          int lo = 0, hi = P.batch.B;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (P.batch.cu[mid] <= tok)
              lo = mid;
            else
              hi = mid;
          }
          const Seq s = load_seq(P, lo, false);
          row_pos = s.keys ? s.pos0 + tok - s.row0 : -1;
        }
        const float row_slope = P.slopes ? P.slopes[head] * kLog2e : 0.f;
        // the warp's queries, scaled per row by a power of two, in fp16: 16 lanes a row, so that loads
        // are of whole lines (a thread per row: 4096 sectors a unit through the L1, 3 us)
        const int64_t row_at = static_cast<int64_t>(u.row0 + tok) * P.sq + head * D;
        const int c16 = lane & 15;
        uint4 qw[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          qw[i] = __ldg(reinterpret_cast<const uint4*>(P.q + __shfl_sync(0xffffffffu, row_at, 2 * i + (lane >> 4))) + c16);
        float row_f = 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t ws[4] = {qw[i].x, qw[i].y, qw[i].z, qw[i].w};
          float mx = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(ws[e] << 16)),
                                 fabsf(__uint_as_float(ws[e] & 0xFFFF0000u))));
#pragma unroll
          for (int of = 1; of < 16; of <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
          const int ex = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu) - 127;
          const int up = mx > 0.f ? max(-126, min(126, 14 - ex)) : 0;
          float qf = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
          float f = __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * P.scale *
                    (SPECIAL && P.cap > 0.f ? 1.0f : kLog2e);
          // a factor >= 0 lets the maximum be taken before it is applied
          if (f < 0.f) f = -f, qf = -qf;
          if (f == 0.f) f = 1.f, qf = 0.f;
          f = fminf(f, 3.0e38f);               // times a score of zero, an infinity would be NaN
          const float both = __shfl_sync(0xffffffffu, f, (lane & 1) << 4);   // of row 2 i + (lane & 1)
          if (lane >> 1 == i) row_f = both;
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[place8<BITS>(2 * e)] = __uint_as_float(ws[e] << 16) * qf;
            v[place8<BITS>(2 * e + 1)] = __uint_as_float(ws[e] & 0xFFFF0000u) * qf;
          }
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = h2_bits(__floats2half2_rn(v[2 * e], v[2 * e + 1]));
          *reinterpret_cast<uint4*>(smem + OFF_Q + hf * 2 * PANEL + chunk_at(32 * quarter + 2 * i + (lane >> 4), c16)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full[hf]);
        float f[4], slope[4];
        int qpos[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          f[x] = __shfl_sync(0xffffffffu, row_f, 8 * x + g);
          slope[x] = -__shfl_sync(0xffffffffu, row_slope, 8 * x + g);
          qpos[x] = __shfl_sync(0xffffffffu, row_pos, 8 * x + g);
        }
        const int qmin = __reduce_min_sync(0xffffffffu, row_pos), qmax = __reduce_max_sync(0xffffffffu, row_pos);
        float ff[4];                         // the scores' factor inside the exponential
        pair_t ff2[4], mneg2[4];             // twice each: it, and the reference taken off
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          ff[x] = SPECIAL ? 1.0f : f[x];
          ff2[x] = pair_of(ff[x], ff[x]);
          mneg2[x] = pair_of(0.f, 0.f);
        }

        for (int j = 0; j < steps; ++j) {
          const int tile = tiles + (j >> 1), ring = tile & 3, b = j & 1, key0 = b * (KT / 2);
          // scores first: they tell that every producer warp has come past the ring's last round, so
          // that a half which skipped units cannot take an older phase of the same parity for this one
          ok = mbar_wait(&bar.s_full[hf][b], (par_s >> b) & 1, spin);
          if (b == 0) ok = ok && mbar_wait(&bar.sc_full[ring], (tile >> 2) & 1, spin);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          par_s ^= 1u << b;
          tc_fence_after();
          const uint32_t t_s = t_s0 + key0;
          // this lane's pairs of scales: keys 8 c + 2 t, + 1
          const pair_t* sk2 = reinterpret_cast<const pair_t*>(s_sk + ring * KT + key0) + t;
          const pair_t* sv2 = reinterpret_cast<const pair_t*>(s_sv + ring * KT + key0) + t;
          const int kpos = tile_pos(P, u, j >> 1) + key0;
          if (SPECIAL && P.cap > 0.f) {
            // capped scores, in log2 units, back to tensor memory
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t w[2][4];
              const float2 sk = floats_of(sk2[4 * c]);
#pragma unroll
              for (int bk = 0; bk < 2; ++bk) tmem_ld_16x256b_x1(t_s + (bk << 20) + 8 * c, w[bk]);
              tmem_ld_wait();
#pragma unroll
              for (int bk = 0; bk < 2; ++bk) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[bk][e] = __float_as_uint(
                      P.cap * tanh_score(__uint_as_float(w[bk][e]) * ((e & 1) ? sk.y : sk.x) *
                                         f[2 * bk + (e >> 1)] * P.inv_cap) * kLog2e);
                tmem_st_16x256b_x1(t_s + (bk << 20) + 8 * c, w[bk]);
              }
            }
            tmem_st_wait();
          }
          // ---- 64 scores (times the key's scale; the row's factor follows), hidden ones -inf
          uint32_t v[2][32];
          tmem_ld_16x256b_x8(t_s, v[0]);
          tmem_ld_16x256b_x8(t_s + (16u << 16), v[1]);
          const uint4 fl = *reinterpret_cast<const uint4*>(s_hid + ring * 8 + 4);
          const uint32_t flags = fl.x | fl.y | fl.z | fl.w;
          const bool edge = flags != 0u || kpos + KT / 2 - 1 > qmin || (P.window > 0 && qmax - kpos >= P.window);
          tmem_ld_wait();
          if (!SPECIAL || P.cap <= 0.f) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const pair_t sk = sk2[4 * c];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mul2u(v[x >> 1][4 * c + 2 * (x & 1)], v[x >> 1][4 * c + 2 * (x & 1) + 1], sk);
            }
          }
          if (SPECIAL && P.slopes != nullptr) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float d0 = static_cast<float>(qpos[x] - kpos - 2 * t), fx = P.cap > 0.f ? 1.0f : f[x];
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t* w = &v[x >> 1][4 * c + 2 * (x & 1)];
                const f2 dist = add2(f2{d0, d0}, f2{-8.0f * c, -8.0f * c - 1.0f});
                const f2 y = fma2(f2{slope[x], slope[x]}, dist,
                                  mul2(f2{__uint_as_float(w[0]), __uint_as_float(w[1])}, f2{fx, fx}));
                w[0] = __float_as_uint(y.x);
                w[1] = __float_as_uint(y.y);
              }
            }
          }
          if (edge) {
            // keys lo .. hi - 1 of the step are visible to a row by position
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int hi = qpos[x] - kpos + 1, lo = P.window > 0 ? hi - P.window : 0;
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const uint32_t seen = (bits_below(hi - 32 * w) & ~bits_below(lo - 32 * w) &
                                       ~s_hid[ring * 8 + (key0 >> 5) + w]) >> (2 * t);
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    uint32_t& y = v[x >> 1][16 * w + 4 * c + 2 * (x & 1) + e];
                    y = (seen & (1u << (8 * c + e))) ? y : 0xFF800000u;
                  }
              }
            }
          }
          // ---- references, and the sums rescaled where one has moved far
          const float2 sve2 = *reinterpret_cast<const float2*>(s_sve + ring * 4 + 2 * b);
          const float sve = fmaxf(sve2.x, sve2.y) - sv_exp, slack = kTop + kSlack - fmaxf(sve, -kReach);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          bool raise = sve > kEnds;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              mx[x] = max3(mx[x], v[x >> 1][4 * c + 2 * (x & 1)], v[x >> 1][4 * c + 2 * (x & 1) + 1]);
            mx[x] = __fmul_rn(mx[x], ff[x]);
            raise |= mx[x] - m[x] > slack;
          }
          if (__any_sync(0xffffffffu, raise)) {
            // lane t works out row t's reference
            auto mine = [&](auto a0, auto a1, auto a2, auto a3) { return t & 2 ? (t & 1 ? a3 : a2) : (t & 1 ? a1 : a0); };
            float seen = sve + sv_exp, shift = 0.f, low = 0.f;
            if (sve > kEnds) {
              // the scales' factor moves, and references with it as far as the sums of exponentials allow
              const float to = seen > kEnds ? seen - kInside : seen < -kEnds ? seen + kInside : 0.f;
              shift = to - sv_exp;
              sv_exp = to;
              const float most = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
              low = fminf(shift, 75.f - __log2f(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)))));
            }
            if (edge) {
              // the keys that a row sees are a run
              const int hi = mine(qpos[0], qpos[1], qpos[2], qpos[3]) - kpos + 1, lo = P.window > 0 ? hi - P.window : 0;
              int e = 0;
#pragma unroll
              for (int w = 0; w < KT / 2; w += 32) {
                const int a = max(lo - w, 0), len = min(hi - w, 32) - a;
                if (len > 0) {
                  const int k = 31 - __clz(len);
                  const uint8_t* run = s_run + 8 * (ring * KT + key0 + w + a) + k;
                  e = max(e, max(run[0], run[8 * (len - (1 << k))]));
                }
              }
              seen = static_cast<float>(e - 126);
            }
            float top[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              top[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
              top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            }
            const float old = mine(m[0], m[1], m[2], m[3]);
            const float now = fmaxf(old - low, mine(top[0], top[1], top[2], top[3]) + fmaxf(seen - sv_exp, -kReach) - kTop);
            const float fa = ex2(old - now), down = ex2(-shift);
            far = sv_exp != 0.f || __any_sync(0xffffffffu, fabsf(now) > kPlain && now > kNone);
            float g4[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              m[x] = __shfl_sync(0xffffffffu, now, (lane & 28) + x);
              g4[x] = __shfl_sync(0xffffffffu, fa, (lane & 28) + x);
              l[x] *= g4[x];
              g4[x] *= down;
              mneg2[x] = pair_of(-m[x], -m[x]);
            }
            if (j > 0) {
              // the product of the step before; its barrier's phase before that was done when these
              // scores came
              ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_full[hf][1 - b], ((par_o >> (1 - b)) & 1) ^ 1, spin));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t w[2][16];
#pragma unroll
                for (int bk = 0; bk < 2; ++bk) tmem_ld_16x256b_x4(t_o + (bk << 20) + 32 * c, w[bk]);
                tmem_ld_wait();
#pragma unroll
                for (int bk = 0; bk < 2; ++bk) {
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    w[bk][e] = __float_as_uint(__uint_as_float(w[bk][e]) * g4[2 * bk + ((e >> 1) & 1)]);
                  tmem_st_16x256b_x4(t_o + (bk << 20) + 32 * c, w[bk]);
                }
              }
              tmem_st_wait();
            }
          }
          // ---- weights
          pair_t sum[4] = {0, 0, 0, 0};
          uint32_t o[2][16];
          // (the common case is compiled by itself: branches inside cost it half its rate)
          auto weights = [&](auto careful) {
            const float svi = !far ? 1.0f : power_of_two(-sv_exp);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const pair_t sv = careful.value ? pair_mul(sv2[4 * c], pair_of(svi, svi)) : sv2[4 * c];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int at = 4 * c + 2 * (x & 1);
                float2 y;
                if (careful.value)             // (never fused by the compiler, which a mul and an add of pairs were)
                  y = make_float2(__fadd_rn(__fmul_rn(__uint_as_float(v[x >> 1][at]), ff[x]), -m[x]),
                                  __fadd_rn(__fmul_rn(__uint_as_float(v[x >> 1][at + 1]), ff[x]), -m[x]));
                else
                  y = floats_of(pair_fma(pair_of(v[x >> 1][at], v[x >> 1][at + 1]), ff2[x], mneg2[x]));
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                const pair_t a = pair_of(e.x, e.y);
                sum[x] = pair_add(sum[x], a);
                float2 w = floats_of(pair_mul(a, sv));
                if (careful.value) {         // a hidden key's scale may be infinite or NaN
                  w.x = e.x == 0.f ? 0.f : w.x;
                  w.y = e.y == 0.f ? 0.f : w.y;
                }
                o[x >> 1][2 * c + (x & 1)] = h2_bits(__floats2half2_rn(w.x, w.y));
              }
            }
          };
          if (!far && !(flags & 2u))
            weights(std::false_type());
          else
            weights(std::true_type());
#pragma unroll
          for (int bk = 0; bk < 2; ++bk) tmem_st_16x128b_x8(t_s + (bk << 20), o[bk]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 s2 = floats_of(sum[x]);
            l[x] = fmaf(s2.x + s2.y, kDown, l[x]);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[hf][b]);
          par_o ^= 1u << b;
        }
        // the last product: its barrier's phase before was done when the last scores came
        if (ok && n > 0) {
          const int b = (steps - 1) & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_full[hf][b], ((par_o >> b) & 1) ^ 1, spin));
          tc_fence_after();
        }
      }
      // a thread per row again
      float lr = 0.f, mr = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const float a = __shfl_sync(0xffffffffu, l[x], 4 * (lane & 7)), c = __shfl_sync(0xffffffffu, m[x], 4 * (lane & 7));
        if (lane >> 3 == x) lr = a, mr = c;
      }
      tiles += n;
      if (!ok) break;
      // ---- out.  Partial results stay at 2^-40 of themselves, their reference 40 higher (large scales might
      // carry them past float32's end), but where small scales might take them past its other end.
      const int pieces = u.pieces, slot = u.slot;
      const bool split = pieces > 1 && !P.shared, live = row < rows;
      const float svr = power_of_two(fmaxf(sv_exp, -126.f));
      mr = lr == 0.f ? -INFINITY : mr + 40.0f;
      if ((split || P.shared) && sv_exp < 0.f) mr -= 40.0f, lr *= 1.0f / kDown;
      const int at = u.base + min(row, rows - 1), tok = at / P.G, head = u.h * P.G + at - tok * P.G;
      const int64_t out_row = static_cast<int64_t>(u.row0 + tok) * P.hq + head;
      float* part_o = nullptr;               // partial results, and this row's place in them
      int64_t part_row = 0;
      if (P.shared) {
        const int64_t to = static_cast<int64_t>(u.piece) * P.batch.T * P.hq + out_row;
        part_o = P.ex_o + static_cast<int64_t>(u.piece) * P.batch.T * P.hq * D;
        part_row = out_row;
        if (active && live) {
          P.ex_ml[2 * to] = mr;
          P.ex_ml[2 * to + 1] = lr;
        }
      } else if (split) {
        float* p = P.tpart + (static_cast<int64_t>(slot) * P.nsplit + u.piece) * (2 * HALF * (D + 2));
        part_o = p;
        part_row = row;
        if (active) {
          p[2 * HALF * D + 2 * row] = live ? mr : -INFINITY;
          p[2 * HALF * D + 2 * row + 1] = live ? lr : 0.f;
        }
      }
      if (active) {
        // through this half's queries, which nothing reads any more, so that 16 lanes store a row's
        // whole lines
        // (a result's 2^-40 in two parts: neither factor leaves float32's range)
        const float inv = part_o ? (sv_exp < 0.f ? 1.0f : kDown) : lr == 0.f ? 0.f : 9.5367432e-07f / lr;
        const float fac = part_o ? svr : svr * 9.5367432e-07f;
        uint8_t* stage = smem + OFF_Q + hf * 2 * PANEL;
        const int lane_row = part_o ? static_cast<int>(part_row) : static_cast<int>(out_row);
        const int passes = part_o ? 2 : 1;
#pragma unroll 1
        for (int pass = 0; pass < passes; ++pass) {
          __syncwarp();
#pragma unroll 1
          for (int c = 2 * pass; c < (part_o ? 2 * pass + 2 : 4); ++c) {
            uint32_t v[32];
            if (n > 0) {
              tmem_ld32(t_o + 32 * c, v);
              tmem_ld_wait();
            }
#pragma unroll
            for (int c8 = 0; c8 < 4; ++c8) {
              float y[8];
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                const float o = __uint_as_float(v[8 * c8 + place8<BITS>(d)]);
                y[d] = n > 0 && lr != 0.f ? o * inv * fac : 0.f;
              }
              if (part_o) {
                const int at = 8 * (c & 1) + 2 * c8;
                *reinterpret_cast<float4*>(stage + chunk_at(r, at)) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(stage + chunk_at(r, at + 1)) = make_float4(y[4], y[5], y[6], y[7]);
              } else {
                uint32_t w[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * d], y[2 * d + 1]);
                  w[d] = *reinterpret_cast<uint32_t*>(&b2);
                }
                *reinterpret_cast<uint4*>(stage + chunk_at(r, 4 * c + c8)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          __syncwarp();
          const int live_rows = min(32, rows - hf * HALF - 32 * quarter);
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            const int q = 2 * i + (lane >> 4);
            const int64_t to = __shfl_sync(0xffffffffu, lane_row, q);
            if (q < live_rows) {
              const uint4 w = *reinterpret_cast<const uint4*>(stage + chunk_at(32 * quarter + q, lane & 15));
              if (part_o)
                *reinterpret_cast<uint4*>(part_o + to * D + 64 * pass + 4 * (lane & 15)) = w;
              else
                *reinterpret_cast<uint4*>(P.out + to * D + 8 * (lane & 15)) = w;
            }
          }
        }
        if (!part_o && live && P.lse)
          P.lse[out_row] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
      }
      if (split) {
        // mbarriers rather than a named barrier: a half that gave up must not leave the other
        // waiting for good
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.parts);
        if (warp == 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bar.parts, splits & 1, spin));
          if (!ok) break;
          if (lane == 0) {
            __threadfence();
            const unsigned seen = atomicAdd(P.tcount + slot, 1u);
            bar.last = seen == static_cast<unsigned>(pieces - 1);
            if (bar.last) P.tcount[slot] = 0;
            mbar_arrive(&bar.joined);
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.joined, splits & 1, spin));
        ++splits;
        if (!ok) break;
        if (bar.last) {
          __threadfence();
          const float* all = P.tpart + static_cast<int64_t>(slot) * P.nsplit * (2 * HALF * (D + 2));
          constexpr int AT_ONCE = 4;       // rows a warp joins at a time: their loads overlap
          for (int q0 = warp * AT_ONCE; q0 < rows; q0 += 8 * AT_ONCE) {
            float M[AT_ONCE], L[AT_ONCE];
            float4 acc[AT_ONCE];
#pragma unroll
            for (int d = 0; d < AT_ONCE; ++d) {
              M[d] = -INFINITY;
              L[d] = 0.f;
              acc[d] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int p = 0; p < pieces; ++p) {
              const float* pp = all + static_cast<int64_t>(p) * (2 * HALF * (D + 2));
              float2 ml[AT_ONCE];
              float4 o[AT_ONCE];
#pragma unroll
              for (int d = 0; d < AT_ONCE; ++d) {
                const int q = min(q0 + d, rows - 1);
                ml[d] = __ldcg(reinterpret_cast<const float2*>(pp + 2 * HALF * D) + q);
                o[d] = __ldcg(reinterpret_cast<const float4*>(pp + q * D) + lane);
              }
#pragma unroll
              for (int d = 0; d < AT_ONCE; ++d) {
                const float nm = fmaxf(M[d], ml[d].x);
                const float fa = M[d] == -INFINITY ? 0.f : ex2(M[d] - nm);
                const float fb = ml[d].x == -INFINITY ? 0.f : ex2(ml[d].x - nm);
                M[d] = nm;
                L[d] = L[d] * fa + ml[d].y * fb;
                acc[d].x = acc[d].x * fa + (fb != 0.f ? o[d].x * fb : 0.f);
                acc[d].y = acc[d].y * fa + (fb != 0.f ? o[d].y * fb : 0.f);
                acc[d].z = acc[d].z * fa + (fb != 0.f ? o[d].z * fb : 0.f);
                acc[d].w = acc[d].w * fa + (fb != 0.f ? o[d].w * fb : 0.f);
              }
            }
#pragma unroll
            for (int d = 0; d < AT_ONCE; ++d) {
              const int q = q0 + d;
              if (q >= rows) continue;
              const int tq = (u.base + q) / P.G, hq_ = u.h * P.G + u.base + q - tq * P.G;
              const int64_t orow = static_cast<int64_t>(u.row0 + tq) * P.hq + hq_;
              const float inv = L[d] == 0.f ? 0.f : 1.0f / L[d];
              __nv_bfloat162 a = __floats2bfloat162_rn(acc[d].x * inv, acc[d].y * inv);
              __nv_bfloat162 b = __floats2bfloat162_rn(acc[d].z * inv, acc[d].w * inv);
              *reinterpret_cast<uint2*>(P.out + orow * D + 4 * lane) =
                  make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
              if (P.lse && lane == 0) P.lse[orow] = L[d] == 0.f ? -INFINITY : (M[d] + log2f(L[d])) * kLn2;
            }
          }
        }
        __syncwarp();                      // bar.last has been read: the next unit's write waits for
      }                                    // every warp's next arrival
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.u_free[k % UNITS]);
    }
  } else if (warp < 12) {
    // ----------------------------------------------------------- widening
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(BITS == 4 ? 64 : 88));
    const int pw = warp - 8, t = lane & 3, b3 = lane >> 2;
    // rows of a warp's load instruction; the two rows of a store phase differ in a bit that the
    // lanes' chunks do not use (see widen_rows)
    const int rsub = BITS == 4 ? ((b3 & 1) << 1) | ((b3 >> 1) & 1) | (b3 & 4) : b3;
    const int wrow = 32 * pw;
    int tiles = 0;
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_full[k % UNITS], (k / UNITS) & 1, spin));
      if (!ok) break;
      const volatile TileUnit& u = ring_u[k % UNITS];
      if (u.rows == 0) break;
      const int n = u.n, h = u.h;
      TileCodes<BITS> kc, vc;
      // of this lane's row, wrow + lane: scales, zero points
      float sk = 0.f, sv = 0.f;
      int kz = 0, vz = 0;
      bool gone = true;
      int64_t grp[2];                      // cache rows of the warp's two groups of 16 in the tile being loaded
      auto pages = [&](int i, int (&pg)[2]) {
        const TileAt at = tile_at(P, u, min(i, n - 1));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int l = at.local + wrow + 16 * j;
          pg[j] = l < at.limit ? at.table[l >> P.pages.lps] : -1;
          if (l < at.limit && (pg[j] < 0 || pg[j] >= P.pages.num_pages)) {
            if (lane == 0 && h == 0) record_status(SQ_ERR_INVALID_ARG);
            pg[j] = -1;
          }
        }
      };
      // every address lies in a page: rows behind the last one are read and hidden, a group without a
      // page reads page 0
      auto load_k = [&](int i, const int (&pg)[2]) {
        const TileAt at = tile_at(P, u, i);
        const int l0 = at.local + wrow, in_page = (1 << P.pages.lps) - 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) grp[j] = group_of(P.pages, max(pg[j], 0), h, (l0 + 16 * j) & in_page);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4* src = reinterpret_cast<const uint4*>(P.pages.kc + (grp[j >> 1] + 8 * (j & 1) + rsub) * RB) + t;
#pragma unroll
          for (int c = 0; c < BITS / 4; ++c) kc.c[j][c] = __ldg(src + 4 * c);
        }
        const int64_t mine = (lane < 16 ? grp[0] : grp[1]) + (lane & 15);
        sk = __ldg(P.pages.ks + mine);
        sv = __ldg(P.pages.vs + mine);
        kz = __ldg(P.pages.kz + mine);
        vz = __ldg(P.pages.vz + mine);
        gone = (lane < 16 ? pg[0] : pg[1]) < 0 || l0 + lane >= at.limit;
      };
      auto load_v = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4* src = reinterpret_cast<const uint4*>(P.pages.vc + (grp[j >> 1] + 8 * (j & 1) + rsub) * RB) + t;
#pragma unroll
          for (int c = 0; c < BITS / 4; ++c) vc.c[j][c] = __ldg(src + 4 * c);
        }
      };
      int pg[2];
      if (n > 0) {
        pages(0, pg);
        load_k(0, pg);
        load_v();
        pages(1, pg);
      }
      for (int i = 0; i < n; ++i, ++tiles) {
        const int st = tiles & 1, ring = tiles & 3;
        const uint32_t par = ((tiles >> 1) & 1) ^ 1;   // a fresh barrier counts as free
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_free[st], par, spin));
        if (!ok) break;
        const int vz_now = vz;
        widen_rows<BITS>(smem + OFF_K + st * 2 * PANEL, kc, kz, wrow, rsub, t);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_full[st]);
        // scales, hidden keys
        s_sk[ring * KT + wrow + lane] = sk;
        s_sv[ring * KT + wrow + lane] = gone ? 0.f : sv;
        const float a = gone ? 0.f : fabsf(sv);
        const bool fine = a <= 3.0e38f;
        // exponents: the largest of the 2^k value scales from this lane's on, a byte for each k of 0 .. 5
        // (infinities and NaN count as zeros)
        uint32_t top = fine ? __float_as_uint(a) >> 23 : 0u;
        uint32_t run[2] = {top, 0u};
#pragma unroll
        for (int k = 1; k < 6; ++k) {
          const uint32_t next = __shfl_down_sync(0xffffffffu, top, 1 << (k - 1));
          if (lane + (1 << (k - 1)) < 32) top = max(top, next);
          run[k >> 2] |= top << (8 * (k & 3));
        }
        *reinterpret_cast<uint2*>(s_run + 8 * (ring * KT + wrow + lane)) = make_uint2(run[0], run[1]);
        const uint32_t hid = __ballot_sync(0xffffffffu, gone), bad = __ballot_sync(0xffffffffu, !fine);
        if (lane == 0) {
          s_sve[ring * 4 + pw] = static_cast<float>(static_cast<int>(top) - 126);
          s_hid[ring * 8 + pw] = hid;
          s_hid[ring * 8 + 4 + pw] = (hid != 0 ? 1u : 0u) | (bad != 0 ? 2u : 0u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sc_full[ring]);
        if (i + 1 < n) load_k(i + 1, pg);
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.v_free[st], par, spin));
        if (!ok) break;
        widen_rows<BITS>(smem + OFF_V + st * 2 * PANEL, vc, vz_now, wrow, rsub, t);
        if (i + 1 < n) {
          load_v();
          pages(i + 2, pg);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_full[st]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.u_free[k % UNITS]);
    }
  } else {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(BITS == 4 ? 64 : 56));
    // one warp per half, which sleeps while its half has nothing to do: a single one that polls both
    // halves' barriers takes issue slots and shared memory from the warps that work.  One copy of its code
    // serves both (with the half a constant of two copies, prompts took 477 us against 438)
    if (warp <= 13) {
      issue_products(warp - 12, P, smem, bar, ring_u);
    } else if (warp == 14) {
      // ------------------------------------------------------------- units
      const int64_t units = P.units;
      int at = 0;
      bool more = true;
      // no streaming kernel follows a call of one long sequence: its lengths are checked here
      if (P.few_rows == 0 && !P.shared && blockIdx.x == 0 && lane == 0) load_seq(P, 0, true);
      const int low_tile = P.shared ? first_shared_tile(P) : 0;
      for (int k = 0; ok && more; ++k) {
        more = k * static_cast<int64_t>(gridDim.x) < units;
        const int64_t x = unit_index(k);
        TileUnit u;
        u.rows = 0;
        if (more && (x >= units || !tile_unit(P, x, low_tile, u))) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_free[at % UNITS], ((at / UNITS) & 1) ^ 1, spin));
        if (!ok) break;
        if (lane == 0) {
          ring_u[at % UNITS] = u;
          mbar_arrive(&bar.u_full[at % UNITS]);
        }
        __syncwarp();
        ++at;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, TILE_TMEM);
  }
}

sq_status launch_tile(const AttnParams& P, int bits, cudaStream_t stream) {
  static std::atomic<bool> allowed[64][4];
  const bool special = P.cap > 0.f || P.slopes != nullptr;
  auto kern = bits == 8 ? (special ? tile_kernel<8, true> : tile_kernel<8, false>)
                        : (special ? tile_kernel<4, true> : tile_kernel<4, false>);
  const int d = host::current_device(), v = (bits == 8 ? 2 : 0) + special;
  cudaError_t e = cudaSuccess;
  if (d < 0 || d >= 64 || !allowed[d][v].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TILE_SMEM);
    if (e != cudaSuccess) return host::cuda_fail("cudaFuncSetAttribute(kv tile)", e);
    if (d >= 0 && d < 64) allowed[d][v].store(true);
  }
  if (P.units < 1) return SQ_OK;
  const int64_t cap = host::num_sms();
  const int grid = static_cast<int>(P.units < cap ? P.units : cap);
  e = host::launch_dependent(kern, grid, TILE_THREADS, TILE_SMEM, stream, P);
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv tile launch", e);
}

}  // namespace paged
}  // namespace sq
