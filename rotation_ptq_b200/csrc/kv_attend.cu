// Attention of a few new tokens per sequence over the paged 4/8-bit cache,
// sm_100a: the streaming kernel.
//
// With rows = (new tokens) x (query heads per KV head) of one KV head, this
// kernel computes, over tiles of 128 keys (32 per warp and step),
//     S^T = C_k Q^T,   s = (S - z_k sum q) sk f_row,   w = exp2(s - m) sv,
//     O^T += (C_v - z_v)^T w
// with C the codes as they are stored, z the zero points and sk, sv the row
// scales, applied in float32.  The products are warp-level m16n8k16 MMAs whose
// operands come straight from the loaded words (a tcgen05 operand would have
// to be widened into swizzled shared memory and synchronised per tile: more
// work than the product).  A code n is used as the fp16 bit pattern n, the
// subnormal n 2^-24: one mask widens two codes; a mask that leaves a nibble
// four bits higher gives 16 n 2^-24, which the query's element (or the
// output's channel) takes back by an exact power of two.  The keys' zero
// points come back once per key and row: 128 terms' sums differ by 2^-24 of
// themselves.  The values' are subtracted before the product (exactly): a sum
// over a long cache of codes that are all positive would lose, against one of
// both signs, what its mean is larger than the result.
//
// What bounds it: issue slots, and the beginning and end of a unit.  Stamps of
// a copy, us from the launch: one sequence of 577 keys, first key 3.6, the last
// CTA's last key 3.9, end 10.7; 16 x 4096, 4.5, 25.8 and 32.0; 48 ragged, 8
// bits, capped, 8.2, 60.7 and 69.0; two of 118 to 131 thousand, 6.1, 74.4 and
// 84.3 (from a last key to its piece's arrival 3, the rest is the join of
// pieces).  16 keys x 128 channels take a warp 392 instructions, a unit's ends
// shared out (374 before rows had normalisers of their own; 592
// with codes widened to whole numbers and loads straight to registers); those two
// documents, 280 MB, take 85 us (158), of which the keys 60, at 4.7 TB/s.
// Loads go through a ring of two slots of 32 keys in shared memory per warp
// (cp.async, no exchange between warps).
//
// Exactness: queries are scaled per row by a power of two that puts the
// largest at 2^14..2^15 and held in fp16 (a bf16 value has 8 significant
// bits, so only values 2^-25 and more below the row's largest lose any);
// products are exact and summed in float32.  Weights are held as the sum of
// two fp16 numbers (22 bits, down to 2^-38 of a row's largest) so that their
// rounding stays below float32 sums'.  With up to 4 rows (PAIR) the product's
// columns 4..7 repeat rows 0..3 and carry the weights' low parts, so that both
// parts take one MMA.
//
// Fragment layout (lane = 4 g + t): the MMA's k order is free as long as both
// operands agree, so lane (g, t) takes row g's t-th contiguous run of codes
// for S, and 16 contiguous dims of key rows 2t, 2t+1, 2t+8, 2t+9 for O.  The
// weights move from S^T's accumulator layout to the B operand by movmatrix.
//
// Work split: the key tiles of all (sequence, row block, KV head) units form
// one list and every CTA takes a contiguous piece of it.  A unit cut between
// CTAs leaves partial (O, m, l) in the workspace; the last CTA to arrive adds
// them in the order of the list, so results do not depend on arrival order.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "kv_attend.cuh"
#include "kv_quant.cuh"
#include "sq_device.cuh"
#include "sq_host.h"

namespace sq {
namespace paged {

constexpr int WARPS = 4, THREADS = 32 * WARPS;
// A row's reference m is its largest score so far less kLift (log2 units), so
// its weights reach 2^kLift and fp16, whose smallest step is 2^-24, holds them
// down to 2^-38 of the largest.  A new maximum may pass the reference by
// kLazy more before the sums are rescaled: weights stay below 2^15.
constexpr float kLift = 14.0f, kLazy = 1.0f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 1 / x of a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float reciprocal(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

__device__ __forceinline__ uint32_t add_bits(uint32_t a, uint32_t b) {
  return h2_bits(__hadd2(bits_h2(a), bits_h2(b)));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A unit: one sequence, block of rows and KV head.
struct Unit {
  Seq s;
  int b, h, row0, rows;                    // row0: first of its (token, head) rows
};

constexpr int kOverhead = 3;               // tiles that a unit's beginning and end cost

template <int BITS, int NT, bool PAIR>
struct Stream {
  static constexpr int R = PAIR ? 4 : 8 * NT;            // rows per unit
  static constexpr int RB = D * BITS / 8;
  static constexpr int DEPTH = 2;                        // ring slots per warp
  // a slot: two groups of 16 keys, each K codes, V codes, K scales, V scales, K zero points,
  // V zero points; behind a unit's keys the ring holds the warp's sums
  static constexpr int V0 = 16 * RB, SC0 = 32 * RB, GROUP = 32 * RB + 160, SLOT = 2 * GROUP;
  static constexpr int RING = DEPTH * SLOT;
  static constexpr int SMEM = WARPS * RING;
  static_assert(R * D * 4 <= RING, "sums in the ring");
  static constexpr int CTAS = NT == 1 ? 3 : 2;

  // Where 16-byte chunk c of key row r lies: rows are permuted inside 128-byte lines so that the
  // lanes of a load phase, two keys apart (V) or one (K), do not share banks.
  static __device__ __forceinline__ int k_at(int r, int c) {
    return BITS == 4 ? r * 64 + c * 16 : r * 128 + ((c ^ ((r & 1) << 2)) << 4);
  }
  static __device__ __forceinline__ int v_at(int r, int c) {
    return BITS == 4 ? (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4)
                     : r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4);
  }

  // Query fragments of the unit's rows, and each of this thread's two columns'
  // factor (log2 units, or plain when the scores are capped), 2^24 aside: a
  // row near bf16's end would carry the product past float32's.
  static __device__ __forceinline__ void load_q(const AttnParams& P, const Unit& u, int g, int t,
                                                uint32_t (&qb)[NT][8][2], float (&qf)[NT][2],
                                                float (&qs)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = PAIR ? g & 3 : 8 * n + g;
      float x[32];
      const bool live = r < u.rows;
      const int row = u.row0 + (live ? r : 0);
      const int tok = row / P.G, head = u.h * P.G + row - tok * P.G;
      const __nv_bfloat16* src = P.q + (u.s.row0 + tok) * P.sq + head * D;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // the lane's run of 32 dims: 32 t.. at 4 bits, 16 t.. and 64 + 16 t.. at 8
        const int d = BITS == 4 ? 32 * t + 8 * c : 16 * t + 8 * (c & 1) + 64 * (c >> 1);
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(src + d));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[8 * c + 2 * e] = __uint_as_float(ws[e] << 16);
          x[8 * c + 2 * e + 1] = __uint_as_float(ws[e] & 0xFFFF0000u);
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) mx = fmaxf(mx, fabsf(x[e]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^(14 - floor(log2 mx)), its exponent kept inside float32's
      const int ex = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu) - 127;
      const int up = mx > 0.f ? max(-126, min(126, 14 - ex)) : 0;
      float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      // a factor >= 0 lets the maximum be taken before it is applied
      float mine = inv * P.scale * (P.cap > 0.f ? 1.0f : kLog2e);
      if (mine < 0.f) mine = -mine, f = -f;
      if (mine == 0.f) mine = 1.f, f = 0.f;
      mine = fminf(mine, 3.0e38f);         // times a score of zero, an infinity would be NaN
      // 4-bit codes of the second register of a pair are 16 n 2^-24
      const float fb = BITS == 4 ? f * 0.0625f : f;
      float sum = 0.f;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        // the pairs that the masks below leave
        const float* y = x + (BITS == 4 ? 8 * (st >> 1) : 4 * st);
        const int i0 = BITS == 4 ? 2 * (st & 1) : 0;
        const int a0 = i0, a1 = BITS == 4 ? i0 + 4 : 1, b0 = BITS == 4 ? i0 + 1 : 2,
                  b1 = BITS == 4 ? i0 + 5 : 3;
        qb[n][st][0] = live ? h2_bits(__floats2half2_rn(y[a0] * f, y[a1] * f)) : 0u;
        qb[n][st][1] = live ? h2_bits(__floats2half2_rn(y[b0] * fb, y[b1] * fb)) : 0u;
        const float2 lo = __half22float2(bits_h2(qb[n][st][0])), hi = __half22float2(bits_h2(qb[n][st][1]));
        sum += (lo.x + lo.y) + (hi.x + hi.y) * (BITS == 4 ? 16.0f : 1.0f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= 5.9604645e-08f;               // codes are n 2^-24
      // the factor of row 8 n + g lives in its lanes; columns 2t, 2t + 1 need rows 2t, 2t + 1
      qs[n][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
      qs[n][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      qf[n][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
      qf[n][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
    }
  }
};

template <int BITS, int NT, bool PAIR>
__global__ void __launch_bounds__(THREADS, Stream<BITS, NT, PAIR>::CTAS) stream_kernel(const AttnParams P) {
  using St = Stream<BITS, NT, PAIR>;
  constexpr int R = St::R, RB = St::RB;
  extern __shared__ __align__(128) uint8_t stream_smem[];
  auto sm_o = [&](int w) { return reinterpret_cast<float(*)[D]>(stream_smem + w * St::RING); };
  __shared__ float sm_m[WARPS][R], sm_l[WARPS][R], sm_f[THREADS], sm_fl[THREADS], sm_top[R];
  __shared__ int64_t sm_scan[2 * WARPS], sm_base;
  __shared__ int sm_b;
  __shared__ bool sm_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = P.G, hkv = P.pages.hkv, B = P.batch.B;
  // a programmatic dependent.  Behind a shared prefix's pass its CTAs begin with the sequences' own keys
  // as that pass's end (it has waited for what was before it), and wait where they join
  if (P.ex_n == 0) griddep_wait();
  griddep_launch_dependents();
  const bool split = P.part != nullptr;

  // ---- the list: this CTA's piece, and the sequence it begins in
  auto count = [&](const Seq& s) {         // units of a sequence
    return s.qlen * G > P.many_rows ? 0ll : static_cast<long long>((s.qlen * G + R - 1) / R) * hkv;
  };
  const int chunk = (B + THREADS - 1) / THREADS, bfirst = tid * chunk, blast = min(B, bfirst + chunk);
  // Few units (a decode step of long sequences): each gets CTAs of its own, as many as share its tiles
  // evenly, since a CTA that ends one unit and begins another pays twice for a unit's beginning and
  // end (6 of 84 us for two 131k documents).  Many: all get equal pieces of the list of tiles, where
  // a unit's beginning and end count as kOverhead tiles (a batch of ragged lengths would else leave
  // the CTAs with the short ones behind: 101 against 62 us).
  int64_t tiles = 0, units = 0;
  bool slots = false;
  int per_slot = 1;
  // places of a unit in the list: slots, or tiles behind kOverhead; a unit without keys still writes zeros
  auto places = [&](const Seq& s) {
    const int n = max(s.tiles(), 1);
    return !split ? 1 : slots ? (n + per_slot - 1) / per_slot : n + kOverhead;
  };
  auto choose = [&]() {
    slots = split && 2 * units <= gridDim.x;
    if (slots) per_slot = static_cast<int>(min(tiles / (gridDim.x - units) + 1, static_cast<int64_t>(1 << 30)));
  };
  auto warp_sum = [&](int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  auto warp_scan = [&](int64_t v) {        // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  int64_t total, base, piece, r0, r1;
  int b;
  // equal pieces but for the last; a unit's pieces belong to consecutive CTAs
  auto cut = [&]() {
    piece = slots ? 1 : (total + gridDim.x - 1) / gridDim.x;
    r0 = piece * blockIdx.x;
    r1 = min(total, r0 + piece);
    if (r0 < r1) return true;
    griddep_wait();                        // this kernel's end tells that of the shared prefix's pass too
    return false;
  };
  if (B <= 32) {
    // every warp by itself, a lane per sequence: no barriers
    const Seq s = load_seq(P, min(lane, B - 1), blockIdx.x == 0 && tid < B);
    const int64_t n = lane < B ? count(s) : 0;
    units = warp_sum(n);
    tiles = warp_sum(n * max(s.tiles(), 1));
    choose();
    const int64_t w = n * places(s), incl = warp_scan(w);
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (!cut()) return;
    b = __ffs(__ballot_sync(0xffffffffu, r0 < incl)) - 1;
    base = __shfl_sync(0xffffffffu, incl - w, b);
  } else {
    for (int q = bfirst; q < blast; ++q) {
      const Seq s = load_seq(P, q, blockIdx.x == 0);
      units += count(s);
      tiles += count(s) * max(s.tiles(), 1);
    }
    units = warp_sum(units);
    tiles = warp_sum(tiles);
    if (lane == 0) {
      sm_scan[warp] = units;
      sm_scan[WARPS + warp] = tiles;
    }
    __syncthreads();
    units = tiles = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      units += sm_scan[w];
      tiles += sm_scan[WARPS + w];
    }
    choose();
    int64_t mine = 0;
    for (int q = bfirst; q < blast; ++q) {
      const Seq s = load_seq(P, q, false);
      mine += count(s) * places(s);
    }
    const int64_t incl = warp_scan(mine);
    __syncthreads();
    if (lane == 31) sm_scan[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += sm_scan[w];
      total += sm_scan[w];
    }
    const int64_t excl = before + incl - mine;
    if (!cut()) return;
    if (r0 >= excl && r0 < excl + mine) {
      int q = bfirst;
      int64_t at = excl;
      for (;; ++q) {
        const Seq s = load_seq(P, q, false);
        const int64_t w = count(s) * places(s);
        if (r0 < at + w) break;
        at += w;
      }
      sm_b = q;
      sm_base = at;
    }
    __syncthreads();
    b = sm_b;
    base = sm_base;
  }

  for (int64_t cur = r0; cur < r1;) {
    Unit u;
    u.s = load_seq(P, b, false);
    const int per = places(u.s), all = u.s.tiles();
    const int64_t wgt = count(u.s) * per;
    if (cur >= base + wgt) {
      base += wgt;
      ++b;
      continue;
    }
    int64_t unit;
    if (wgt >> 31 == 0)
      unit = static_cast<uint32_t>(cur - base) / static_cast<uint32_t>(per);
    else
      unit = (cur - base) / per;
    const int i0 = static_cast<int>((cur - base) - unit * per);
    const int i1 = static_cast<int>(min(static_cast<int64_t>(per), i0 + (r1 - cur)));
    const int64_t u0 = base + unit * per;  // the unit's place in the list
    cur += i1 - i0;
    // this CTA's tiles of the unit, and the CTAs that have any
    int first = 0, last = all;
    int64_t c0 = 0, c1 = 0;
    if (slots) {
      first = static_cast<int>(static_cast<int64_t>(all) * i0 / per);
      last = static_cast<int>(static_cast<int64_t>(all) * i1 / per);
      c0 = u0;
      c1 = u0 + per - 1;
    } else if (split) {
      const int lead = per - max(all, 1);
      first = max(i0 - lead, 0);
      last = i1 - lead;
      if (last <= first) continue;         // the unit's overhead alone
      last = min(last, all);
      if (first > 0 || last < all) {
        c0 = (u0 + lead) / piece;
        c1 = (u0 + per - 1) / piece;
      }
    }
    const bool whole = c0 == c1;
    u.b = b;
    u.row0 = wgt >> 31 == 0 ? static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(hkv))
                            : static_cast<int>(unit / hkv);
    u.h = static_cast<int>(unit - static_cast<int64_t>(u.row0) * hkv);
    u.row0 *= R;
    u.rows = min(R, u.s.qlen * G - u.row0);

    // ---- the way of 32 keys into the ring: the shared prefix's tiles that are this CTA's (where no
    // other kernel takes them), then the own
    const uint8_t* ring = stream_smem + warp * St::RING;
    const uint32_t ring32 = smem_u32(ring);
    // lanes 0..3 fetch a group's K scales, 4..7 its V scales, 8 and 9 its zero points
    const uint8_t* extra = reinterpret_cast<const uint8_t*>(lane < 4 ? P.pages.ks : P.pages.vs) + 16 * (lane & 3);
    if (lane == 8) extra = P.pages.kz;
    if (lane == 9) extra = P.pages.vz;
    const int extra_step = lane < 8 ? 4 : 1;
    const int in_page = (1 << P.pages.lps) - 1;
    int local, end, limit, kshift, pg[2];
    const int32_t* table;
    // pages of both groups of 16, -1: no keys
    auto pages_of = [&](int row, int (&to)[2]) {
      to[0] = row < end ? __ldg(table + (row >> P.pages.lps)) : -1;
      to[1] = row + 16 < end ? __ldg(table + ((row + 16) >> P.pages.lps)) : -1;
    };
    unsigned there = 0;                    // bits 2 slot + group: it holds keys
    auto fetch = [&](int from, const int (&pages)[2], int slot) {
      there &= ~(3u << (2 * slot));
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        const int row = from + 16 * gr;
        if (row < end) {
          if (pages[gr] < 0 || pages[gr] >= P.pages.num_pages) {
            if (lane == 0) record_status(SQ_ERR_INVALID_ARG);
          } else {
            const int64_t grp = group_of(P.pages, pages[gr], u.h, row & in_page);
            const uint32_t dst = ring32 + slot * St::SLOT + gr * St::GROUP;
            const uint8_t* kc = P.pages.kc + grp * RB + 16 * lane;
            const uint8_t* vc = P.pages.vc + grp * RB + 16 * lane;
            constexpr int CPR = RB / 16, RPI = 32 / CPR;         // chunks per row, rows per instruction
#pragma unroll
            for (int j = 0; j < 16 / RPI; ++j) {
              const int rw = j * RPI + lane / CPR, c = lane % CPR;
              cp_async16(dst + St::k_at(rw, c), kc + 512 * j);
              cp_async16(dst + St::V0 + St::v_at(rw, c), vc + 512 * j);
            }
            if (lane < 10) cp_async16(dst + St::SC0 + 16 * lane, extra + grp * extra_step);
            there |= 1u << (2 * slot + gr);
          }
        }
      }
      cp_async_commit();
    };
    auto begin = [&](int seg) {            // a segment's first two slots on their way
      const int t0 = seg ? u.s.ot0 + max(first - u.s.pn, 0) : u.s.pt0 + first;
      const int t1 = seg ? u.s.ot0 + last - u.s.pn : u.s.pt0 + min(last, u.s.pn);
      limit = seg ? u.s.len : P.prefix_len;
      kshift = seg ? P.prefix_len : 0;
      table = seg ? P.batch.table + static_cast<int64_t>(u.b) * P.batch.width : P.prefix_table;
      end = min(limit, t1 * TILE);
      local = t0 * TILE + 32 * warp;
      int next[2];
      pages_of(local, pg);
      pages_of(local + TILE, next);
      fetch(local, pg, 0);
      fetch(local + TILE, next, 1);
      pages_of(local + 2 * TILE, pg);
    };
    const int seg0 = first < u.s.pn ? 0 : 1;
    begin(seg0);

    uint32_t qb[NT][8][2];
    float qf[NT][2], qs[NT][2];
    St::load_q(P, u, g, t, qb, qf, qs);
    // this thread's columns: rows 8 n + 2 t + {0, 1}
    int qpos[NT][2];
    float slope[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = min(PAIR ? 2 * (t & 1) + e : 8 * n + 2 * t + e, u.rows - 1);
        const int tok = (u.row0 + r) / G;
        qpos[n][e] = u.s.pos0 + tok;
        slope[n][e] = P.slopes ? P.slopes[u.h * G + u.row0 + r - tok * G] * kLog2e : 0.f;
      }
    const int qmin = u.s.pos0 + u.row0 / G, qmax = u.s.pos0 + (u.row0 + u.rows - 1) / G;

    float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    const bool special = P.cap > 0.f || P.slopes != nullptr;
    // The rows' factors wait for the exponential's fused multiply-add, unless the scores are capped or
    // sloped, so large (kPlain) that the multiply-add's own rounding would tell its result from the
    // maximum's, or a row's factor leaves float32: then they are applied to the scores.
    bool factored = special;
#pragma unroll
    for (int n = 0; n < NT; ++n) factored = factored || qf[n][0] > 1.0e30f || qf[n][1] > 1.0e30f;
    factored = __any_sync(0xffffffffu, factored);
    float ff[NT][2];                       // the factor inside the exponential
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) ff[n][e] = factored ? 1.f : qf[n][e] * 16777216.0f;
    // 1 / a power of two above the value scales that the row has seen so far: a hidden key's, however
    // large, takes no bits from the weights of a row
    float svi[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) svi[n][0] = svi[n][1] = 8.507059e37f;  // 2^126

#pragma unroll 1
    for (int seg = seg0; seg < 2; ++seg) {
      if (seg != seg0) begin(seg);
      for (int slot = 0; local < end; local += TILE, slot ^= 1) {
        cp_async_wait<St::DEPTH - 1>();
        __syncwarp();
        const unsigned have = (there >> (2 * slot)) & 3u;
        if (have) {
          const uint8_t* sl = ring + slot * St::SLOT;
          const int kpos = kshift + local;
          // ---- S^T = C_k Q^T: [group][n][0], [1] key g; [2], [3] key g + 8; columns 2t, 2t + 1
          float sc[2][NT][4], sk[2][2], sv[2][2], kz[2][2];
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const uint8_t* x = sl + gr * St::GROUP;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              sk[gr][hf] = reinterpret_cast<const float*>(x + St::SC0)[g + 8 * hf];
              sv[gr][hf] = reinterpret_cast<const float*>(x + St::SC0)[16 + g + 8 * hf];
              kz[gr][hf] = static_cast<float>(x[St::SC0 + 128 + g + 8 * hf]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[gr][n][e] = 0.f;
#pragma unroll
            for (int c = 0; c < BITS / 4; ++c) {
              const uint4 a4 = *reinterpret_cast<const uint4*>(x + St::k_at(g, t + 4 * c));
              const uint4 b4 = *reinterpret_cast<const uint4*>(x + St::k_at(g + 8, t + 4 * c));
              const uint32_t wa[4] = {a4.x, a4.y, a4.z, a4.w}, wb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                if (BITS == 4) {
                  const uint32_t a8 = wa[w] >> 8, b8 = wb[w] >> 8;
                  const uint32_t f0[4] = {wa[w] & 0x000F000Fu, wb[w] & 0x000F000Fu,
                                          wa[w] & 0x00F000F0u, wb[w] & 0x00F000F0u};
                  const uint32_t f1[4] = {a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u,
                                          b8 & 0x00F000F0u};
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    mma16816(sc[gr][n], f0, qb[n][2 * w][0], qb[n][2 * w][1]);
                    mma16816(sc[gr][n], f1, qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
                  }
                } else {
                  const uint32_t f0[4] = {__byte_perm(wa[w], 0u, 0x4140u), __byte_perm(wb[w], 0u, 0x4140u),
                                          __byte_perm(wa[w], 0u, 0x4342u), __byte_perm(wb[w], 0u, 0x4342u)};
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma16816(sc[gr][n], f0, qb[n][4 * c + w][0], qb[n][4 * c + w][1]);
                }
              }
            }
          }
          // ---- scores; without a cap or slopes the row's factor waits for the exponential
          const bool plain = !special && have == 3u && local + 32 <= limit && kpos + 31 <= qmin &&
                             (P.window == 0 || qmax - kpos < P.window);
#pragma unroll
          for (int gr = 0; gr < 2; ++gr)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sc[gr][n][e] = fmaf(-kz[gr][e >> 1], qs[n][e & 1], sc[gr][n][e]) * sk[gr][e >> 1];
          auto apply = [&]() {
#pragma unroll
            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[gr][n][e] = sc[gr][n][e] * qf[n][e & 1] * 16777216.0f;
          };
          if (factored) apply();
          const float all = fmaxf(fmaxf(fabsf(sv[0][0]), fabsf(sv[0][1])), fmaxf(fabsf(sv[1][0]), fabsf(sv[1][1])));
          float sva[NT][2];                // the largest value scale that the row sees of this lane's keys
#pragma unroll
          for (int n = 0; n < NT; ++n) sva[n][0] = sva[n][1] = plain ? all : 0.f;
          if (!plain) {
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int hf = e >> 1, c = e & 1;
                  float x = sc[gr][n][e];
                  const int dist = qpos[n][c] - (kpos + 16 * gr + g + 8 * hf);
                  if (special) {
                    if (P.cap > 0.f) x = P.cap * tanh_score(x * P.inv_cap) * kLog2e;
                    x = fmaf(-slope[n][c], static_cast<float>(dist), x);
                  }
                  const bool seen = dist >= 0 && (P.window == 0 || dist < P.window) &&
                                    local + 16 * gr + g + 8 * hf < limit && ((have >> gr) & 1u);
                  sc[gr][n][e] = seen ? x : -INFINITY;
                  sva[n][c] = fmaxf(sva[n][c], seen ? fabsf(sv[gr][hf]) : 0.f);
                }
              // rows behind the last key, and a group that is not there, hold anything
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (local + 16 * gr + g + 8 * hf >= limit || !((have >> gr) & 1u)) sv[gr][hf] = 0.f;
            }
          }
          // ---- references: rescale only when a maximum has moved far
          float mx[NT][2];
          bool raise = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              mx[n][c] = fmaxf(fmaxf(sc[0][n][c], sc[0][n][2 + c]), fmaxf(sc[1][n][c], sc[1][n][2 + c])) *
                         ff[n][c];
              raise |= mx[n][c] - m[n][c] > kLift + kLazy || sva[n][c] * svi[n][c] > 1.0f;
            }
          if (__any_sync(0xffffffffu, raise)) {
            bool large = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float svmax = 0.f;         // infinities and NaN set none
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float a = fabsf(sv[j >> 1][j & 1]);
                  svmax = fmaxf(svmax, a <= 3.0e38f && sc[j >> 1][n][2 * (j & 1) + c] != -INFINITY ? a : 0.f);
                }
#pragma unroll
                for (int of = 4; of < 32; of <<= 1)
                  svmax = fmaxf(svmax, __shfl_xor_sync(0xffffffffu, svmax, of));
                // 1 / a power of two above svmax, between 2^-126 and 2^126
                const int e2 = max(1, min(253, static_cast<int>(__float_as_uint(svmax) >> 23) + 1));
                const float nsvi = fminf(svi[n][c], __uint_as_float(static_cast<uint32_t>(254 - e2) << 23));
                const float down = nsvi * reciprocal(svi[n][c]);
                svi[n][c] = nsvi;
                float top = mx[n][c];
#pragma unroll
                for (int of = 4; of < 32; of <<= 1)
                  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, of));
                // (float32's steps may be wider than the lift)
                top = fmaxf(top - (top - kLift) > kLift + kLazy ? top : top - kLift, m[n][c]);
                large |= top > kPlain || (top < -kPlain && top > -INFINITY);
                const float f = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - top);
                m[n][c] = top;
                l[n][c] *= f;
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) {
                  o[n][i8][c] *= f * down;
                  o[n][i8][2 + c] *= f * down;
                }
              }
            if (!factored && __any_sync(0xffffffffu, large)) {
              apply();
              factored = true;
#pragma unroll
              for (int n = 0; n < NT; ++n) ff[n][0] = ff[n][1] = 1.f;
            }
          }
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            // ---- weights, as fp16 pairs (high, low), to the B operand's layout
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float p[4], w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                p[e] = ex2(fmaf(sc[gr][n][e], ff[n][e & 1], -m[n][e & 1]));
                w[e] = p[e] * (sv[gr][e >> 1] * svi[n][e & 1]);
              }
              if (!plain) {                // no reference yet, or a hidden key's infinite scale
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (sc[gr][n][e] == -INFINITY) p[e] = 0.f;
                  if (p[e] == 0.f) w[e] = 0.f;
                }
              }
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const float w0 = w[2 * hf], w1 = w[2 * hf + 1];
                l[n][0] += p[2 * hf];
                l[n][1] += p[2 * hf + 1];
                const __half2 hi = __floats2half2_rn(w0, w1);
                const float2 back = __half22float2(hi);
                const uint32_t lo = h2_bits(__floats2half2_rn(w0 - back.x, w1 - back.y));
                if (PAIR) {
                  ph[n][hf] = transpose8x8(t < 2 ? h2_bits(hi) : lo);
                } else {
                  ph[n][hf] = transpose8x8(h2_bits(hi));
                  pl[n][hf] = transpose8x8(lo);
                }
              }
            }
            // ---- O^T += (C_v - z_v)^T w: dims 16 g + 2 i + {0, 1} in m-tile i
            const uint8_t* x = sl + gr * St::GROUP;
            uint32_t vz[2];                // zero points of keys 2t, 2t + 1 (+ 8): fp16 -z 2^-24
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              vz[hf] = __byte_perm(reinterpret_cast<const uint16_t*>(x + St::SC0 + 144)[t + 4 * hf], 0u, 0x4140u) |
                       0x80008000u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t va[8], vb[8];       // 8 dims of key pairs (2t, 2t+1) and (2t+8, 2t+9)
#pragma unroll
              for (int pr = 0; pr < 2; ++pr) {
                uint32_t(&dst)[8] = pr ? vb : va;
                if (BITS == 4) {
                  const int at = 8 * (g & 1) + 4 * half;
                  const uint32_t vz16 = ((vz[pr] & 0x000F000Fu) << 4) | 0x80008000u;
                  const uint32_t a = *reinterpret_cast<const uint32_t*>(
                      x + St::V0 + St::v_at(2 * t + 8 * pr, g >> 1) + at);
                  const uint32_t bb = *reinterpret_cast<const uint32_t*>(
                      x + St::V0 + St::v_at(2 * t + 1 + 8 * pr, g >> 1) + at);
#pragma unroll
                  for (int hw = 0; hw < 2; ++hw) {
                    const uint32_t mix = __byte_perm(a, bb, hw ? 0x7632u : 0x5410u), m8 = mix >> 8;
                    dst[4 * hw] = add_bits(mix & 0x000F000Fu, vz[pr]);
                    dst[4 * hw + 1] = add_bits(mix & 0x00F000F0u, vz16);
                    dst[4 * hw + 2] = add_bits(m8 & 0x000F000Fu, vz[pr]);
                    dst[4 * hw + 3] = add_bits(m8 & 0x00F000F0u, vz16);
                  }
                } else {
                  const uint2 a2 = *reinterpret_cast<const uint2*>(
                      x + St::V0 + St::v_at(2 * t + 8 * pr, g) + 8 * half);
                  const uint2 b2 = *reinterpret_cast<const uint2*>(
                      x + St::V0 + St::v_at(2 * t + 1 + 8 * pr, g) + 8 * half);
#pragma unroll
                  for (int hw = 0; hw < 2; ++hw) {
                    const uint32_t a = hw ? a2.y : a2.x, bb = hw ? b2.y : b2.x;
                    const uint32_t lo = __byte_perm(a, bb, 0x5140u), hi = __byte_perm(a, bb, 0x7362u);
                    dst[4 * hw] = add_bits(__byte_perm(lo, 0u, 0x4140u), vz[pr]);
                    dst[4 * hw + 1] = add_bits(__byte_perm(lo, 0u, 0x4342u), vz[pr]);
                    dst[4 * hw + 2] = add_bits(__byte_perm(hi, 0u, 0x4140u), vz[pr]);
                    dst[4 * hw + 3] = add_bits(__byte_perm(hi, 0u, 0x4342u), vz[pr]);
                  }
                }
              }
#pragma unroll
              for (int i4 = 0; i4 < 4; ++i4) {
                const uint32_t a[4] = {va[2 * i4], va[2 * i4 + 1], vb[2 * i4], vb[2 * i4 + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  mma16816(o[n][4 * half + i4], a, ph[n][0], ph[n][1]);
                  if (!PAIR) mma16816(o[n][4 * half + i4], a, pl[n][0], pl[n][1]);
                }
              }
            }
          }
          __syncwarp();
        }
        fetch(local + 2 * TILE, pg, slot);
        pages_of(local + 3 * TILE, pg);
      }
      cp_async_wait<0>();
      __syncwarp();
    }

    // ---- the warps' results into shared memory.  Sums that large scales might carry past float32's end
    // before they are divided stand at 2^-40 of themselves, their reference 40 higher.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        const float svr = reciprocal(svi[n][c]), back = 16777216.0f * (svr >= 1.0f ? 9.094947e-13f : 1.0f);
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) {
          l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], of);
        }
        if (g == 0 && r < R) {
          sm_m[warp][r] = svr >= 1.0f ? m[n][c] + 40.0f : m[n][c];
          sm_l[warp][r] = svr >= 1.0f ? l[n][c] * 9.094947e-13f : l[n][c];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x = o[n][i][c], y = o[n][i][2 + c];
          if (PAIR) {                      // the low parts' columns
            x += __shfl_down_sync(0xffffffffu, x, 2);
            y += __shfl_down_sync(0xffffffffu, y, 2);
          }
          x = x * back * svr;
          y = y * (BITS == 4 ? 0.0625f * back : back) * svr;
          if (r < R) *reinterpret_cast<float2*>(&sm_o(warp)[r][16 * g + 2 * i]) = make_float2(x, y);
        }
      }
    __syncthreads();
    // thread tid owns dim tid of every row
    const int part = 2 * blockIdx.x + (u0 >= r0 ? 1 : 0);
    constexpr int PART = R * (D + 2);
    float acc[R], mm[R], ll[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_m[w][r]);
      acc[r] = ll[r] = 0.f;
      mm[r] = M;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = sm_m[w][r] == -INFINITY ? 0.f : ex2(sm_m[w][r] - M);
        if (f != 0.f) acc[r] = fmaf(f, sm_o(w)[r][tid], acc[r]);
        ll[r] = fmaf(f, sm_l[w][r], ll[r]);
      }
    }
    bool finish = whole;
    // adds n pieces (ml(j, r): reference and sum; o(j, r): this thread's dim) to (acc, mm, ll): the
    // largest reference first, then 128 / R pieces' factors at a time by one thread each, so that
    // every load but the factors' is independent
    auto join = [&](int n, auto ml, auto out) {
      constexpr int STEP = THREADS / R, AHEAD = 32 / R;
      const int jr = tid % R, jq = tid / R;
      if (n <= AHEAD) {                    // few pieces: everything at once
        float2 q[AHEAD][R];
        float po[AHEAD][R];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            q[k][r] = ml(min(k, n - 1), r);
            po[k][r] = out(min(k, n - 1), r);
          }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float x = mm[r];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) x = fmaxf(x, q[k][r].x);
          float f = mm[r] == -INFINITY ? 0.f : ex2(mm[r] - x);
          acc[r] = f != 0.f ? acc[r] * f : 0.f;
          ll[r] *= f;
          mm[r] = x;
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            f = k >= n || q[k][r].x == -INFINITY ? 0.f : ex2(q[k][r].x - x);
            if (f != 0.f) acc[r] = fmaf(f, po[k][r], acc[r]);
            ll[r] = fmaf(f, q[k][r].y, ll[r]);
          }
        }
        return;
      }
      const float2 mine = jq < n ? ml(jq, jr) : make_float2(-INFINITY, 0.f);
      float top = mine.x;
      for (int q = jq + STEP; q < n; q += STEP) top = fmaxf(top, ml(q, jr).x);
      sm_f[tid] = top;
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x = mm[r];
        for (int k = 0; k < STEP; ++k) x = fmaxf(x, sm_f[k * R + r]);
        const float f = mm[r] == -INFINITY ? 0.f : ex2(mm[r] - x);
        acc[r] = f != 0.f ? acc[r] * f : 0.f;
        ll[r] *= f;
        mm[r] = x;
        if (tid == r) sm_top[r] = x;
      }
      for (int q0 = 0; q0 < n; q0 += STEP) {
        __syncthreads();
        const int q = q0 + jq;
        float f = 0.f, fl = 0.f;
        if (q < n) {
          const float2 v = q0 == 0 ? mine : ml(q, jr);
          f = v.x == -INFINITY ? 0.f : ex2(v.x - sm_top[jr]);
          fl = f * v.y;
        }
        sm_f[tid] = f;
        sm_fl[tid] = fl;
        __syncthreads();
        const int cnt = min(STEP, n - q0);
        for (int k0 = 0; k0 < cnt; k0 += AHEAD) {
          float po[AHEAD][R];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int r = 0; r < R; ++r) po[k][r] = out(q0 + min(k0 + k, cnt - 1), r);
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
            if (k0 + k < cnt) {
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const float w = sm_f[(k0 + k) * R + r];
                if (w != 0.f) acc[r] = fmaf(w, po[k][r], acc[r]);
                ll[r] += sm_fl[(k0 + k) * R + r];
              }
            }
        }
      }
      __syncthreads();
    };
    if (!whole) {
      float* p = P.part + static_cast<int64_t>(part) * PART;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        p[r * D + tid] = acc[r];
        if (tid == 0) {
          p[R * D + r] = mm[r];
          p[R * D + R + r] = ll[r];
        }
      }
      __syncthreads();
      if (tid == 0) {
        __threadfence();                   // the whole block's writes, which the barrier has ordered before
        const unsigned seen = atomicAdd(P.count + c0, 1u);
        sm_last = seen == static_cast<unsigned>(c1 - c0);
        if (sm_last) P.count[c0] = 0;
      }
      __syncthreads();
      finish = sm_last;
      if (finish) {
        __threadfence();
#pragma unroll
        for (int r = 0; r < R; ++r) mm[r] = -INFINITY, ll[r] = acc[r] = 0.f;
        auto place = [&](int j) {
          const int64_t c = c0 + j;
          return P.part + (2 * c + (u0 >= c * piece ? 1 : 0)) * PART;
        };
        join(static_cast<int>(c1 - c0) + 1,
             [&](int j, int r) {
               const float* p = place(j) + R * D + r;
               return make_float2(__ldcg(p), __ldcg(p + R));
             },
             [&](int j, int r) { return __ldcg(place(j) + r * D + tid); });
      }
    }
    if (finish) {
      int64_t row[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int rr = min(r, u.rows - 1), tok = (u.row0 + rr) / G;
        row[r] = static_cast<int64_t>(u.s.row0 + tok) * P.hq + u.h * G + u.row0 + rr - tok * G;
      }
      if (P.ex_n > 0) {
        // the shared prefix's part of the rows, in pieces (the pass may have run beside this kernel so far)
        griddep_wait();
        const int64_t step = P.batch.T * P.hq;
        join(P.ex_n,
             [&](int j, int r) {           // r is not known to the compiler here
               const int rr = min(r, u.rows - 1), tok = (u.row0 + rr) / G;
               const int64_t at = static_cast<int64_t>(u.s.row0 + tok) * P.hq + u.h * G + u.row0 + rr - tok * G;
               return __ldcg(reinterpret_cast<const float2*>(P.ex_ml) + j * step + at);
             },
             [&](int j, int r) { return __ldcg(P.ex_o + (j * step + row[r]) * D + tid); });
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r < u.rows) {
          const float y = ll[r] == 0.f ? 0.f : acc[r] / ll[r];
          P.out[row[r] * D + tid] = __float2bfloat16_rn(y);
          if (P.lse && tid == r)
            P.lse[row[r]] = ll[r] == 0.f ? -INFINITY : (mm[r] + log2f(ll[r])) * kLn2;
        }
      }
    }
    __syncthreads();                       // sm_* are free for the next unit
  }
}

namespace {

// The counters' share of a workspace: the same for every variant, so that no
// variant's partial results lie where another expects zeros.
constexpr size_t kCountBytes = 16384;
constexpr int kMaxGrid = kCountBytes / 4;

using StreamFn = void (*)(AttnParams);
struct StreamKernel {
  StreamFn fn;
  int rows, smem;
};

// kind: 0 up to 4 rows a unit, 1 up to 8, 2 up to 16.
template <int BITS>
StreamKernel stream_variant(int kind) {
  if (kind == 0) return {stream_kernel<BITS, 1, true>, 4, Stream<BITS, 1, true>::SMEM};
  if (kind == 1) return {stream_kernel<BITS, 1, false>, 8, Stream<BITS, 1, false>::SMEM};
  return {stream_kernel<BITS, 2, false>, 16, Stream<BITS, 2, false>::SMEM};
}
StreamKernel stream_of(int bits, int kind) {
  return bits == 4 ? stream_variant<4>(kind) : stream_variant<8>(kind);
}

// CTAs that the device holds at once; the first call on a device also allows the kernel its
// shared memory.
int stream_grid(int bits, int kind) {
  static std::atomic<int> cache[64][6];
  const int d = host::current_device(), v = kind + (bits == 4 ? 0 : 3);
  if (d >= 0 && d < 64 && cache[d][v].load() > 0) return cache[d][v].load();
  const StreamKernel k = stream_of(bits, kind);
  int per_sm = 0;
  if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k.fn, THREADS, k.smem) != cudaSuccess ||
      per_sm < 1) {
    (void)cudaGetLastError();
    per_sm = 1;
  }
  const int grid = host::num_sms() * per_sm < kMaxGrid ? host::num_sms() * per_sm : kMaxGrid;
  if (d >= 0 && d < 64) cache[d][v].store(grid);
  return grid;
}

// Sequences of up to this many rows (new tokens x query heads per KV head) go to the streaming kernel
// (in units of 16), longer ones to the tile kernel, whose 128 rows a half cost the same however few of
// them live.  4-bit, 4000 keys, streaming against tile, us: 32 rows of 1, 4, 16 sequences 29 / 28,
// 36 / 44, 85 / 103; 48 rows 30 / 34, 52 / 46, 122 / 102.  With 4 KV heads instead of 8, 1, 4, 16, 48 sequences
// at 4 bits, 32 rows 33 / 27, 30 / 35, 54 / 59, 130 / 184 (8 bits 33 / 28, 30 / 34, 56 / 69, 130 / 223), 64 rows
// 29 / 34, 37 / 41, 89 / 86, 228 / 182 (8 bits 29 / 35, 38 / 39, 91 / 107, 226 / 223), 128 rows 29 / 50, 54 / 48,
// 158 / 87, 423 / 183.  Where there are few units streaming would still win above kFewRows, 48 rows of a single
// KV head at all of these (31 / 34, 28 / 38, 35 / 40, 55 / 58): the tile kernel's work is cut by places, not keys.
constexpr int kFewRows = 32;
// A shared prefix is read once for the batch (by the tile kernel, whose partial results the streaming
// kernel joins) while no sequence has more rows than kSharedRows - longer ones fill the tile kernel's
// rows by themselves - and the streaming kernel's tiles over the prefix, for each sequence anew, would
// come to kSharedTiles an SM.  4-bit, us, streaming against shared: 16 single tokens behind 4096 keys
// 38 / 42, behind 10000 67 / 52; 32 behind 2000 42 / 43, behind 4096 60 / 44; 64 behind 700 44 / 55,
// behind 2000 65 / 55; 5 new tokens each, 6 sequences behind 2000 39 / 47, 32 behind 2000 108 / 89.  8-bit:
// 16 single tokens behind 4096 39 / 39, behind 10000 68 / 45; 32 behind 2000 44 / 37, behind 4096 60 / 43; 64 behind
// 700 43 / 51, behind 2000 65 / 54; 6 behind 10000 35 / 43; 5 new tokens each, 6 behind 4096 56 / 53, behind 10000
// 97 / 58, 16 behind 2000 64 / 50, 32 behind 700 84 / 73: where the rule is wrong, it is by a quarter at most.
// Under a window only the prefix's last keys count: either side reads no others.
constexpr int kSharedRows = 128;
constexpr int kSharedTiles = 30;
constexpr size_t kSharedBytes = size_t{1} << 30;          // of partial results: larger batches stream
constexpr int kTileRows = 256;
constexpr size_t kPartFloats = static_cast<size_t>(kTileRows) * (D + 2);

// share: whether a shared prefix may have a pass of its own (without: a workspace's size where a window rules it out).
AttnPlan make_plan(int64_t T, int hq, int hkv, int B, int max_q, int64_t keys, int prefix_len,
                   int window, int bits, bool have_ws, bool share = true) {
  AttnPlan p{};
  const int64_t G = hq / hkv, rows = G * max_q;
  const int sms = host::num_sms();
  p.kind = rows <= 4 ? 0 : rows <= 8 ? 1 : 2;
  const int64_t per_unit = stream_of(bits, p.kind).rows;
  // rows of the prefix that a sequence without keys of its own sees under the window
  const int64_t seen = window > 0 ? std::min<int64_t>(prefix_len, static_cast<int64_t>(window) + max_q) : prefix_len;
  p.shared = share && have_ws && B > 1 && prefix_len > 0 && rows <= kSharedRows &&
             B * ((rows + per_unit - 1) / per_unit) * hkv * ((seen + TILE - 1) / TILE) >=
                 static_cast<int64_t>(kSharedTiles) * sms &&
             static_cast<size_t>(T) * hq * D * 4 <= kSharedBytes;
  p.tile = !p.shared && rows > kFewRows;
  p.stream = p.shared || !p.tile || B > 1;
  p.tile_split = 1;
  size_t at = 2 * kCountBytes;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  if (p.stream)
    p.part = take(static_cast<size_t>(stream_grid(bits, p.kind)) * 2 * stream_of(bits, p.kind).rows * (D + 2) * 4);
  if (p.shared) {
    const int64_t units = (T * G + kTileRows - 1) / kTileRows * hkv, tiles = (seen + 127) / 128;
    int64_t s = sms / units;
    if (s > (tiles + 1) / 2) s = (tiles + 1) / 2;
    p.tile_split = static_cast<int>(s < 1 ? 1 : s);
    p.tile_units = units * p.tile_split;
    p.ex_o = take(static_cast<size_t>(p.tile_split) * T * hq * D * 4);
    p.ex_ml = take(static_cast<size_t>(p.tile_split) * T * hq * 2 * 4);
  } else if (p.tile) {
    const int64_t slots = (T * G / kTileRows + B) * hkv, tiles = (keys + prefix_len + 127) / 128;
    int64_t s = have_ws ? sms / slots : 1;
    if (s > (tiles + 1) / 2) s = (tiles + 1) / 2;
    if (s < 1 || slots > static_cast<int64_t>(kCountBytes / 4)) s = 1;
    p.tile_split = static_cast<int>(s);
    p.tile_units = slots * s;
    if (s > 1) p.tpart = take(static_cast<size_t>(slots) * s * kPartFloats * 4);
  }
  p.bytes = at;
  return p;
}

// Held over a call's launches, so that no other thread's call of the same stream comes between them: the
// streaming kernel joins what the prefix pass right before it left in the workspace, and leaves out its
// own first wait because that pass has made it.  Streams that share an entry only wait for one another's
// launches; the default stream's two handles are one stream.
std::mutex& launch_order(cudaStream_t stream) {
  static std::mutex order[64];
  uintptr_t h = reinterpret_cast<uintptr_t>(stream == nullptr ? cudaStreamLegacy : stream);
  h ^= h >> 16;
  return order[(h ^ (h >> 6)) & 63];
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int hq, int hkv, int B, int max_q, int64_t keys,
                                 int prefix_len, int bits) {
  // for any window
  return std::max(make_plan(T, hq, hkv, B, max_q, keys, prefix_len, 0, bits, true).bytes,
                  make_plan(T, hq, hkv, B, max_q, keys, prefix_len, 0, bits, true, false).bytes);
}

sq_status run_attention(const void* q, int64_t q_stride, int64_t T, int hq,
                        const sq_kv_pages& pages, const int32_t* prefix_table, int prefix_len,
                        const int32_t* table, int width, const int32_t* cu, const int32_t* lengths,
                        int B, int max_q, const sq_score_rule& rule, void* out, float* lse,
                        void* ws, size_t ws_bytes, cudaStream_t stream) {
  AttnParams P{};
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.sq = q_stride;
  P.pages = Pages{pages.k_codes, pages.k_scale, pages.k_zero, pages.v_codes, pages.v_scale,
                  pages.v_zero, pages.num_pages, 0, pages.hkv};
  while ((1 << P.pages.lps) < pages.page_size) ++P.pages.lps;
  P.batch = Batch{table, cu, lengths, width, B, T};
  P.prefix_table = prefix_table;
  P.prefix_len = prefix_len;
  P.hq = hq;
  P.G = hq / pages.hkv;
  P.scale = rule.scale;
  P.cap = rule.softcap;
  P.inv_cap = rule.softcap > 0.f ? std::min(1.0f / rule.softcap, 3.0e38f) : 0.f;
  P.window = rule.window;
  P.slopes = rule.slopes;
  P.out = static_cast<__nv_bfloat16*>(out);
  P.lse = lse;
  P.spin_limit = host::spin_limit();
  const int64_t keys = static_cast<int64_t>(width) * pages.page_size;
  AttnPlan plan = make_plan(T, hq, pages.hkv, B, max_q, keys, prefix_len, rule.window, pages.bits, true);
  const bool have = ws && ws_bytes >= plan.bytes;
  if (!have) plan = make_plan(T, hq, pages.hkv, B, max_q, keys, prefix_len, rule.window, pages.bits, false);
  uint8_t* base = static_cast<uint8_t*>(ws);
  P.many_rows = plan.tile ? kFewRows : 0x7fffffff;
  P.few_rows = plan.stream ? kFewRows : 0;
  P.shared = plan.shared;
  P.nsplit = plan.tile_split;
  P.units = plan.tile_units;
  if (have) {
    P.count = reinterpret_cast<unsigned*>(base);
    P.tcount = reinterpret_cast<unsigned*>(base + kCountBytes);
    P.part = reinterpret_cast<float*>(base + plan.part);
    P.tpart = reinterpret_cast<float*>(base + plan.tpart);
  }
  if (plan.shared) {
    P.ex_o = reinterpret_cast<float*>(base + plan.ex_o);
    P.ex_ml = reinterpret_cast<float*>(base + plan.ex_ml);
  }
  std::lock_guard<std::mutex> together(launch_order(stream));
  if (plan.tile || plan.shared) {
    const sq_status st = launch_tile(P, pages.bits, stream);
    if (st != SQ_OK) return st;
  }
  if (!plan.stream) return SQ_OK;
  P.ex_n = plan.shared ? plan.tile_split : 0;
  const int grid = stream_grid(pages.bits, plan.kind);
  const StreamKernel k = stream_of(pages.bits, plan.kind);
  const cudaError_t e = host::launch_dependent(k.fn, grid, THREADS, k.smem, stream, P);
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv attention launch", e);
}

}  // namespace paged
}  // namespace sq
