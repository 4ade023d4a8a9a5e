// Attention of many rows over the paged 4/8-bit cache, sm_100a: the tile
// kernel on tcgen05.
//
// A unit is up to 256 rows (token, query head of one KV head) in two halves of
// 128, and a run of 128-key tiles.  Per half and tile
//     S = Q K_int^T            (tensor memory, f32; Q and codes exact in fp16), in two steps of 64 keys
//     y = S sk,  p = exp2(y f_row - m),  P = fp16(p sv)      (tensor memory)
//     O += P V_int             (A from tensor memory, f32)
// with K_int, V_int the codes less their zero points.  The row scales sk and
// sv stay outside the products, so fp16 operands lose nothing; P is rounded
// once to 11 bits, an eighth of what the bf16 output's own rounding may lose.
//
// Warps: 0-3 and 4-7 softmax of half 0 and 1 (a thread per row: no exchange
// between lanes), 8-11 widen codes from global memory into swizzled shared
// memory, 12 issues the products, 13 works out the units.  Each half has two buffers of 64
// scores: the products of a step run while the softmax of the step before does.
//
// Two rows of work: a sequence's own rows over what it sees (splits of a
// unit's tiles are joined by the last CTA to arrive, in order), or, for a
// shared prefix, all sequences' rows over the prefix's tiles, whose partial
// results (O, m, l) the streaming kernel joins with each sequence's own part.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "kv_attend.cuh"
#include "sq_device.cuh"
#include "sq_host.h"

namespace sq {
namespace paged {

constexpr int KT = 128;                    // keys per tile
constexpr int HALF = 128;                  // rows per half
constexpr int TILE_THREADS = 16 * 32;    // warps 14 and 15 fill the last group
constexpr int UNITS = 3;                   // unit records in flight
constexpr int PANEL = 128 * 128;           // bytes of 128 rows x 64 fp16
constexpr int OFF_Q = 0;                   // [half][2 panels]
constexpr int OFF_K = OFF_Q + 4 * PANEL;   // [stage][2 panels]
constexpr int OFF_V = OFF_K + 4 * PANEL;
constexpr int OFF_SK = OFF_V + 4 * PANEL;  // float [4][KT]
constexpr int OFF_SV = OFF_SK + 4 * KT * 4;
constexpr int OFF_HID = OFF_SV + 4 * KT * 4;   // uint32 [4][8]: 4 words of hidden keys, 4 of flags
constexpr int OFF_SVM = OFF_HID + 128;         // float [4][4]: largest value scale of 32 keys
constexpr int OFF_BARS = OFF_SVM + 64;
constexpr int OFF_UNITS = OFF_BARS + 512;      // TileUnit [UNITS]
constexpr int TILE_SMEM = OFF_UNITS + UNITS * 128 + 1024;
constexpr uint32_t TILE_TMEM = 512;        // S [half][buffer] of 64 columns, O [half] of 128
constexpr uint32_t IDESC_S = idesc_f16(128, KT / 2, false, false);
constexpr uint32_t IDESC_O = idesc_f16(128, 128, false, true);

struct TileBars {
  uint64_t k_full[2], v_full[2], k_free[2], v_free[2], sc_full[4];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2];        // s, p, o: [half][buffer]
  uint64_t parts, joined, drain;           // partial results written; who joins them is known
  uint64_t u_full[UNITS], u_free[UNITS];
  uint32_t tmem, last;
};
static_assert(sizeof(TileBars) <= 512, "barriers");

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// A unit as every role sees it.  Warp 13 works them out and hands them on in a ring of records in
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

// Unit `x` of this launch; false if it is empty.
__device__ __forceinline__ bool tile_unit(const AttnParams& P, int64_t x, TileUnit& u) {
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
    u.pt0 = 0;
    u.pn = (P.prefix_len - 1) / KT + 1;
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

// Bits 0 .. n - 1, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// (a, b) *= (x, y), floats held in registers of tensor-memory transfers.
__device__ __forceinline__ void mul2u(uint32_t& a, uint32_t& b, float x, float y) {
  const f2 r = mul2(f2{__uint_as_float(a), __uint_as_float(b)}, f2{x, y});
  a = __float_as_uint(r.x);
  b = __float_as_uint(r.y);
}

// ------------------------------------------------------------ widening

template <int BITS>
struct TileCodes {                         // a producer lane's share of one operand: 4 rows
  uint4 c[4][BITS / 4];
};

template <int BITS>
__device__ __forceinline__ void widen_rows(uint8_t* dst, const TileCodes<BITS>& v,
                                           const int (&zero)[4], int warp_row, int rsub, int t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = warp_row + 8 * j + rsub;
    const __half2 z1 = __half2half2(__int2half_rn(-1024 - zero[j]));
    uint8_t* line = dst + row * 128;
    if (BITS == 4) {
      const __half2 z16 = __half2half2(__int2half_rn(-64 - zero[j]));
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

template <int BITS>
__global__ void __launch_bounds__(TILE_THREADS, 1) tile_kernel(const AttnParams P) {
  constexpr int RB = D * BITS / 8;
  extern __shared__ uint8_t tile_smem_raw[];
  uint8_t* smem = tile_smem_raw + ((1024u - (smem_u32(tile_smem_raw) & 1023u)) & 1023u);
  float* s_sk = reinterpret_cast<float*>(smem + OFF_SK);
  float* s_sv = reinterpret_cast<float*>(smem + OFF_SV);
  uint32_t* s_hid = reinterpret_cast<uint32_t*>(smem + OFF_HID);
  float* s_svm = reinterpret_cast<float*>(smem + OFF_SVM);
  TileBars& bar = *reinterpret_cast<TileBars*>(smem + OFF_BARS);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t spin = P.spin_limit;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.k_free[i], 1);
      mbar_init(&bar.v_free[i], 1);
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
    mbar_init(&bar.drain, 1);
    for (int i = 0; i < UNITS; ++i) {
      mbar_init(&bar.u_full[i], 1);
      mbar_init(&bar.u_free[i], 13);
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
  TileUnit* ring_u = reinterpret_cast<TileUnit*>(smem + OFF_UNITS);
  bool ok = true;

  // registers, of the 512 x 128 that the block is launched with: 128 x (2 x 152 + 104 + 104)
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(152));
    const int hf = warp >> 2, quarter = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t t_s0 = lane_base + hf * 128, t_o = lane_base + 256 + hf * 128;
    const int r = 32 * quarter + lane;     // row within the half
    int tiles = 0, mine = 0, splits = 0;   // tiles seen by the CTA, steps of this half; joins
    const bool special = P.cap > 0.f || P.slopes != nullptr;
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_full[k % UNITS], (k / UNITS) & 1, spin));
      if (!ok) break;
      const volatile TileUnit& u = ring_u[k % UNITS];
      const int rows = u.rows, n = u.n, steps = u.steps;
      if (rows == 0) break;
      const bool active = hf * HALF < rows;
      const int row = hf * HALF + r;
      float f = 1.f, m = -INFINITY, l = 0.f, svr = 0.f, mneg = 0.f;
      bool far = true;
      if (active) {
        const int at = u.base + min(row, rows - 1), tok = at / P.G, head = u.h * P.G + at - tok * P.G;
        int qpos = u.pos0 + tok;
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
          qpos = s.keys ? s.pos0 + tok - s.row0 : -1;
        }
        const float slope = P.slopes ? P.slopes[head] * kLog2e : 0.f;
        // this row's query, scaled by a power of two, in fp16
        const uint4* src = reinterpret_cast<const uint4*>(P.q + (u.row0 + tok) * P.sq + head * D);
        uint4 qw[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) qw[c] = __ldg(src + c);
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t ws[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(ws[e] << 16)),
                                 fabsf(__uint_as_float(ws[e] & 0xFFFF0000u))));
        }
        const int ex = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu) - 127;
        const int up = mx > 0.f ? max(-126, min(126, 14 - ex)) : 0;
        float qf = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
        f = __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * P.scale *
            (P.cap > 0.f ? 1.0f / P.cap : kLog2e);
        // f >= 0 lets the maximum be taken before it is applied
        if (f < 0.f) f = -f, qf = -qf;
        if (f == 0.f) f = 1.f, qf = 0.f;
        uint8_t* dst = smem + OFF_Q + hf * 2 * PANEL + r * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t ws[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[place8<BITS>(2 * e)] = __uint_as_float(ws[e] << 16) * qf;
            v[place8<BITS>(2 * e + 1)] = __uint_as_float(ws[e] & 0xFFFF0000u) * qf;
          }
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = h2_bits(__floats2half2_rn(v[2 * e], v[2 * e + 1]));
          *reinterpret_cast<uint4*>(dst + (c >> 3) * PANEL + (((c & 7) ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full[hf]);
        const float ff = special ? 1.0f : f;

        for (int j = 0; j < steps; ++j, ++mine) {
          const int tile = tiles + (j >> 1), ring = tile & 3, key0 = (j & 1) * (KT / 2), buf = mine & 1;
          // scores first: they tell that every producer warp has come past the ring's last round, so
          // that a half which skipped units cannot take an older phase of the same parity for this one
          ok = mbar_wait(&bar.s_full[hf][buf], (mine >> 1) & 1, spin);
          if (ok && key0 == 0) ok = mbar_wait(&bar.sc_full[ring], (tile >> 2) & 1, spin);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t t_s = t_s0 + buf * (KT / 2);
          const float4* sk4 = reinterpret_cast<const float4*>(s_sk + ring * KT + key0);
          const float4* sv4 = reinterpret_cast<const float4*>(s_sv + ring * KT + key0);
          const int rel = qpos - tile_pos(P, u, j >> 1) - key0;          // distance to the step's first key
          if (special) {
            // capped or sloped scores, in log2 units, back to tensor memory
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[16];
              tmem_ld16(t_s + 16 * c, v);
              tmem_ld_wait();
              const float d0 = static_cast<float>(rel - 16 * c);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 s = sk4[4 * c + e];
                const float sk[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  float y = __uint_as_float(v[4 * e + d]) * sk[d] * f;
                  if (P.cap > 0.f) y = P.cap * kLog2e * tanh_score(y);
                  v[4 * e + d] = __float_as_uint(fmaf(-slope, d0 - static_cast<float>(4 * e + d), y));
                }
              }
              tmem_st16(t_s + 16 * c, v);
            }
            tmem_st_wait();
          }
          // ---- 64 scores (times the key's scale; the row's factor follows), hidden ones -inf; the
          // common case is compiled by itself: branches inside cost it half its rate
          uint32_t v[2][32];
          tmem_ld32(t_s, v[0]);
          tmem_ld32(t_s + 32, v[1]);
          // keys lo .. hi - 1 of the step are visible to this row by position
          const int hi = rel + 1, lo = P.window > 0 ? hi - P.window : 0;
          const uint32_t flags = s_hid[ring * 8 + 4] | s_hid[ring * 8 + 5] | s_hid[ring * 8 + 6] |
                                 s_hid[ring * 8 + 7];
          const bool general = special || __any_sync(0xffffffffu, hi < KT / 2 || lo > 0 || flags != 0u);
          tmem_ld_wait();
          auto scale = [&]() {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 s = sk4[8 * c + e];
                mul2u(v[c][4 * e], v[c][4 * e + 1], s.x, s.y);
                mul2u(v[c][4 * e + 2], v[c][4 * e + 3], s.z, s.w);
              }
          };
          if (!special) scale();
          if (general) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t seen = bits_below(hi - 32 * c) & ~bits_below(lo - 32 * c) &
                                    ~s_hid[ring * 8 + (key0 >> 5) + c];
#pragma unroll
              for (int e = 0; e < 32; ++e) v[c][e] = (seen & (1u << e)) ? v[c][e] : 0xFF800000u;
            }
          }
          // ---- references, and the sums rescaled where one has moved far
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int d = 0; d < 4; ++d)
              mx4[d] = fmaxf(mx4[d], fmaxf(__uint_as_float(v[d >> 1][16 * (d & 1) + 2 * e]),
                                           __uint_as_float(v[d >> 1][16 * (d & 1) + 2 * e + 1])));
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * ff;
          const float4 sm4 = *reinterpret_cast<const float4*>(s_svm + ring * 4);
          const float svmax = fmaxf(fmaxf(sm4.x, sm4.y), fmaxf(sm4.z, sm4.w));
          const bool raise = mx > m + 15.0f || svmax > svr;
          if (__any_sync(0xffffffffu, raise)) {
            const int e2 = max(1, min(253, static_cast<int>(__float_as_uint(svmax) >> 23) + 1));
            const float nsv = fmaxf(svr, __uint_as_float(static_cast<uint32_t>(e2) << 23));
            const float down = svr > 0.f ? svr / nsv : 0.f;
            svr = nsv;
            const float nm = fmaxf(m, mx - 14.0f);
            const float fa = m == -INFINITY ? 0.f : ex2(m - nm);
            m = nm;
            l *= fa;
            // exp2(s - m) / svr is one exponential while both its factors are far from float32's
            // ends; otherwise 1 / svr is applied by itself
            far = svr > 1.1529215e18f || svr < 8.6736174e-19f;          // 2^60, 2^-60
            mneg = m == -INFINITY ? 0.f : -m;
            if (!far) mneg -= static_cast<float>(static_cast<int>(__float_as_uint(svr) >> 23) - 127);
            if (j > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_full[hf][(mine - 1) & 1], ((mine - 1) >> 1) & 1, spin));
              if (!ok) break;
              tc_fence_after();
              const float g = fa * down;
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t w[16];
                tmem_ld16(t_o + 16 * c, w);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * g);
                tmem_st16(t_o + 16 * c, w);
              }
              tmem_st_wait();
            }
          }
          // ---- weights
          const f2 f2f{ff, ff}, f2m{mneg, mneg};
          f2 sum{0.f, 0.f};
          auto weights = [&](auto careful) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                f2 a = fma2(f2{__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])}, f2f, f2m);
                a = f2{ex2(a.x), ex2(a.y)};
                sum = add2(sum, a);
                v[c][2 * e] = __float_as_uint(a.x);
                v[c][2 * e + 1] = __float_as_uint(a.y);
              }
              uint32_t some = 0xffffffffu;
              if (careful.value) {           // a hidden key's scale may be infinite or NaN
                some = 0;
                const float svi = !far ? 1.0f : svr > 0.f ? 1.0f / svr : 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  some |= (__uint_as_float(v[c][e]) == 0.f ? 0u : 1u) << e;
                  v[c][e] = __float_as_uint(__uint_as_float(v[c][e]) * svi);
                }
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 s = sv4[8 * c + e];
                mul2u(v[c][4 * e], v[c][4 * e + 1], s.x, s.y);
                mul2u(v[c][4 * e + 2], v[c][4 * e + 3], s.z, s.w);
              }
              if (careful.value) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[c][e] = (some & (1u << e)) ? v[c][e] : 0u;
              }
              uint32_t o[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = h2_bits(__floats2half2_rn(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])));
              tmem_st16(t_s + 16 * c, o);
            }
          };
          if (!far && !(flags & 2u))
            weights(std::false_type());
          else
            weights(std::true_type());
          l += (sum.x + sum.y) * (far ? 1.0f : svr);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[hf][buf]);
        }
        // one barrier per buffer: the product two steps back, the last one on the same barrier, is done
        // once the scores after it are there
        if (ok && n > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_full[hf][(mine - 1) & 1], ((mine - 1) >> 1) & 1, spin));
          tc_fence_after();
        }
      }
      tiles += n;
      if (!ok) break;
      // ---- out
      const int pieces = u.pieces, slot = u.slot;
      const bool split = pieces > 1 && !P.shared, live = row < rows;
      const int at = u.base + min(row, rows - 1), tok = at / P.G, head = u.h * P.G + at - tok * P.G;
      const int64_t out_row = static_cast<int64_t>(u.row0 + tok) * P.hq + head;
      float* part_o = nullptr;
      if (P.shared) {
        const int64_t to = static_cast<int64_t>(u.piece) * P.batch.T * P.hq + out_row;
        part_o = P.ex_o + to * D;
        if (active && live) {
          P.ex_ml[2 * to] = m;
          P.ex_ml[2 * to + 1] = l;
        }
      } else if (split) {
        float* p = P.tpart + (static_cast<int64_t>(slot) * P.nsplit + u.piece) * (2 * HALF * (D + 2));
        part_o = p + row * D;
        if (active) {
          p[2 * HALF * D + 2 * row] = live ? m : -INFINITY;
          p[2 * HALF * D + 2 * row + 1] = live ? l : 0.f;
        }
      }
      if (active) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          if (n > 0) {
            tmem_ld32(t_o + 32 * c, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int c8 = 0; live && c8 < 4; ++c8) {
            float y[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              const float o = __uint_as_float(v[8 * c8 + place8<BITS>(d)]);
              y[d] = n > 0 && l != 0.f ? o * svr : 0.f;
            }
            if (part_o) {
              float4* dst = reinterpret_cast<float4*>(part_o + 32 * c + 8 * c8);
              dst[0] = make_float4(y[0], y[1], y[2], y[3]);
              dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              uint32_t w[4];
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * d] * inv, y[2 * d + 1] * inv);
                w[d] = *reinterpret_cast<uint32_t*>(&b2);
              }
              *reinterpret_cast<uint4*>(P.out + out_row * D + 32 * c + 8 * c8) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
        if (!part_o && live && P.lse)
          P.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(104));
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
      int kz[4], vz[4];
      float sc[4];                         // lane t = 0: key scale; t = 1: value scale
      uint32_t hidden = 0;
      int64_t grp[4];                      // cache rows of the tile being loaded (-1: hidden)
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
      auto load_k = [&](int i, const int (&pg)[2]) {
        const TileAt at = tile_at(P, u, i);
        hidden = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int l = at.local + wrow + 8 * j + rsub;
          const int page = pg[j >> 1];
          const bool gone = page < 0 || l >= at.limit;
          grp[j] = gone ? -1 : group_of(P.pages, page, h, l & ((1 << P.pages.lps) - 1));
          hidden |= static_cast<uint32_t>(gone) << (8 * j + rsub);
          sc[j] = 0.f;
          kz[j] = vz[j] = 0;
#pragma unroll
          for (int c = 0; c < BITS / 4; ++c) kc.c[j][c] = make_uint4(0u, 0u, 0u, 0u);
          if (!gone) {
            const uint4* src = reinterpret_cast<const uint4*>(P.pages.kc + grp[j] * RB) + t;
#pragma unroll
            for (int c = 0; c < BITS / 4; ++c) kc.c[j][c] = __ldg(src + 4 * c);
            kz[j] = __ldg(P.pages.kz + grp[j]);
            vz[j] = __ldg(P.pages.vz + grp[j]);
            if (t < 2) sc[j] = __ldg((t ? P.pages.vs : P.pages.ks) + grp[j]);
          }
        }
      };
      auto load_v = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int c = 0; c < BITS / 4; ++c) vc.c[j][c] = make_uint4(0u, 0u, 0u, 0u);
          if (grp[j] >= 0) {
            const uint4* src = reinterpret_cast<const uint4*>(P.pages.vc + grp[j] * RB) + t;
#pragma unroll
            for (int c = 0; c < BITS / 4; ++c) vc.c[j][c] = __ldg(src + 4 * c);
          }
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
        int vz_now[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) vz_now[j] = vz[j];
        widen_rows<BITS>(smem + OFF_K + st * 2 * PANEL, kc, kz, wrow, rsub, t);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_full[st]);
        // scales, hidden keys
        float svm = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = wrow + 8 * j + rsub;
          if (t == 0) s_sk[ring * KT + row] = sc[j];
          if (t == 1) {
            s_sv[ring * KT + row] = sc[j];
            const float a = fabsf(sc[j]);
            svm = fmaxf(svm, a <= 3.0e38f ? a : 0.f);
            bad |= !(a <= 3.0e38f);
          }
        }
        svm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(svm)));
        const uint32_t hid = __reduce_or_sync(0xffffffffu, hidden);
        const bool any_bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
          s_svm[ring * 4 + pw] = svm;
          s_hid[ring * 8 + pw] = hid;
          s_hid[ring * 8 + 4 + pw] = (hid != 0 ? 1u : 0u) | (any_bad ? 2u : 0u);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 12) {
    int tiles = 0, qs = 0, cnt = 0;          // qs: bit h, half h's parity; cnt: 2 bits, its steps so far
    const uint64_t q_desc = desc_sw128(smem_u32(smem + OFF_Q)), k_desc = desc_sw128(smem_u32(smem + OFF_K)),
                   v_desc = desc_sw128_mn(smem_u32(smem + OFF_V), PANEL, 1024);
    for (int k = 0; ok; ++k) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.u_full[k % UNITS], (k / UNITS) & 1, spin));
      if (!ok) break;
      const volatile TileUnit& u = ring_u[k % UNITS];
      const int rows = u.rows, n = u.n, steps = u.steps;
      if (rows == 0) break;
      const int halves = rows > HALF ? 2 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.u_free[k % UNITS]);
      // descriptors advance by constants in their low word (addresses / 16): few registers
      auto scores = [&](int h, int j, int buf) {
        if (lane == 0) {
          const int stage = (tiles + (j >> 1)) & 1;
          const uint64_t a = q_desc + ((h * 2 * PANEL) >> 4),
                         b = k_desc + ((stage * 2 * PANEL + (j & 1) * (PANEL / 2)) >> 4);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t off = ((s >> 2) * PANEL + (s & 3) * 32) >> 4;
            mma_f16_ss(tmem + h * 128 + buf * (KT / 2), a + off, b + off, IDESC_S, s > 0);
          }
          mma_commit(&bar.s_full[h][buf]);
          if (h == halves - 1 && ((j & 1) || j == steps - 1)) mma_commit(&bar.k_free[stage]);
        }
        __syncwarp();
      };
      for (int h = 0; h < halves && ok; ++h) {
        ok = mbar_wait(&bar.q_full[h], (qs >> h) & 1, spin);
        qs ^= 1 << h;
      }
      if (ok && n > 0) ok = mbar_wait(&bar.k_full[tiles & 1], (tiles >> 1) & 1, spin);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // two steps of scores ahead: a half's next scores are there when its softmax ends
#pragma unroll 1
      for (int j = 0; j < min(steps, 2); ++j)
#pragma unroll 1
        for (int h = 0; h < halves; ++h) scores(h, j, ((cnt >> (2 * h)) + j) & 1);
      for (int j = 0; j < steps && ok; ++j) {
        const int tile = tiles + (j >> 1);
#pragma unroll 1
        for (int h = 0; h < halves && ok; ++h) {
          const int c = (cnt >> (2 * h)) & 3, buf = c & 1;
          ok = mbar_wait(&bar.p_full[h][buf], c >> 1, spin);
          cnt = (cnt & ~(3 << (2 * h))) | (((c + 1) & 3) << (2 * h));
          if (ok && h == 0 && !(j & 1)) ok = mbar_wait(&bar.v_full[tile & 1], (tile >> 1) & 1, spin);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t b = v_desc + (((tile & 1) * 2 * PANEL + (j & 1) * (PANEL / 2)) >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_f16_ts(tmem + 256 + h * 128, tmem + h * 128 + buf * (KT / 2) + 8 * s, b + s * (2048 >> 4),
                         IDESC_O, j > 0 || s > 0);
            mma_commit(&bar.o_full[h][buf]);
            if (h == halves - 1 && ((j & 1) || j == steps - 1)) mma_commit(&bar.v_free[tile & 1]);
          }
          __syncwarp();
          if (j + 2 < steps) {
            if (h == 0 && !(j & 1)) {
              ok = __all_sync(0xffffffffu,
                              mbar_wait(&bar.k_full[(tile + 1) & 1], ((tile + 1) >> 1) & 1, spin));
              if (!ok) break;
              tc_fence_after();
            }
            scores(h, j + 2, buf);
          }
        }
      }
      tiles += n;
    }
    // no product may still write the tensor memory freed below
    if (lane == 0) {
      mma_commit(&bar.drain);
      mbar_wait(&bar.drain, 0, 0);
    }
    __syncwarp();
    } else if (warp == 13) {
      // ------------------------------------------------------------- units
      const int64_t units = P.units;
      int at = 0;
      bool more = true;
      // no streaming kernel follows a call of one long sequence: its lengths are checked here
      if (P.few_rows == 0 && !P.shared && blockIdx.x == 0 && lane == 0) load_seq(P, 0, true);
      for (int k = 0; ok && more; ++k) {
        more = k * static_cast<int64_t>(gridDim.x) < units;
        const int64_t x = unit_index(k);
        TileUnit u;
        u.rows = 0;
        if (more && (x >= units || !tile_unit(P, x, u))) continue;
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
  auto kern = bits == 8 ? tile_kernel<8> : tile_kernel<4>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TILE_SMEM);
  if (e != cudaSuccess) return host::cuda_fail("cudaFuncSetAttribute(kv tile)", e);
  if (P.units < 1) return SQ_OK;
  const int64_t cap = host::num_sms();
  const int grid = static_cast<int>(P.units < cap ? P.units : cap);
  kern<<<grid, TILE_THREADS, TILE_SMEM, stream>>>(P);
  e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv tile launch", e);
}

}  // namespace paged
}  // namespace sq
