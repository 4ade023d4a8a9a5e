// Attention of a few new tokens per sequence over the paged 4/8-bit cache,
// sm_100a: the streaming kernel.
//
// With rows = (new tokens) x (query heads per KV head) of one KV head, this
// kernel computes, over tiles of 64 keys,
//     S^T = K_int Q^T,   s = S sk f_row,   w = exp2(s - m) sv,   O^T += V_int^T w
// where K_int, V_int are codes less zero points (integers in [-255, 255],
// exact in fp16), sk and sv the row scales, applied in float32.  Its time is
// that of streaming the cache: 4 x 16-row-code products per loaded byte are
// far below the tensor pipe, so the products are warp-level m16n8k16 MMAs
// whose operands come straight from the loaded words without a trip through
// shared memory (a tcgen05 operand would have to be widened into swizzled
// shared memory and synchronised per tile: more work than the product).
//
// Exactness: queries are scaled per row by a power of two that puts the
// largest at 2^14..2^15 and held in fp16 (a bf16 value has 8 significant
// bits, so only values 2^-29 and more below the row's largest lose any);
// products are exact and summed in float32.  Weights are held as the sum of
// two fp16 numbers (22 bits, down to 2^-38 of a row's largest) so that their
// rounding stays below float32 sums'.
//
// Fragment layout (lane = 4 g + t): the MMA's k order is free as long as both
// operands agree, so lane (g, t) takes row g's t-th contiguous run of codes
// for S, and 16 contiguous dims of key rows 2t, 2t+1, 2t+8, 2t+9 for O.  The
// weights move from S^T's accumulator layout to the B operand by movmatrix.
//
// Work split: the key tiles of all (sequence, row block, KV head) units form
// one list and every CTA takes an equal contiguous piece.  A unit cut between
// CTAs leaves partial (O, m, l) in the workspace; the last CTA to arrive adds
// them in the order of the list, so results do not depend on arrival order.
#include <cuda_bf16.h>
#include <math.h>

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

template <int BITS>
struct KFrag {                             // a lane's codes of one key row: 32
  uint4 c[BITS / 4];
};
template <int BITS>
struct VFrag {                             // 16 dims of one key row
  uint2 c[BITS / 4];
};

// A unit: one sequence, block of rows and KV head.
struct Unit {
  Seq s;
  int b, h, row0, rows;                    // row0: first of its (token, head) rows
};

template <int BITS, int NT>
struct Stream {
  static constexpr int R = 8 * NT;         // rows per unit
  static constexpr int RB = D * BITS / 8;
  static constexpr int KW = 2 * BITS;      // words of a lane's K run

  // Query fragments of the unit's rows, and each of this thread's two columns'
  // factor (log2 units, or plain when the scores are capped).
  static __device__ __forceinline__ void load_q(const AttnParams& P, const Unit& u, int g, int t,
                                                uint32_t (&qb)[NT][8][2], float (&qf)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
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
      const float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        // the pairs that widen_nibbles / widen_bytes leave
        const float* y = x + (BITS == 4 ? 8 * (st >> 1) : 4 * st);
        const int i0 = BITS == 4 ? 2 * (st & 1) : 0;
        const int a0 = i0, a1 = BITS == 4 ? i0 + 4 : 1, b0 = BITS == 4 ? i0 + 1 : 2,
                  b1 = BITS == 4 ? i0 + 5 : 3;
        qb[n][st][0] = live ? h2_bits(__floats2half2_rn(y[a0] * f, y[a1] * f)) : 0u;
        qb[n][st][1] = live ? h2_bits(__floats2half2_rn(y[b0] * f, y[b1] * f)) : 0u;
      }
      // the factor of row 8 n + g lives in its lanes; columns 2t, 2t + 1 need rows 2t, 2t + 1
      const float mine = inv * P.scale * (P.cap > 0.f ? 1.0f / P.cap : kLog2e);
      qf[n][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
      qf[n][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
    }
  }
};

template <int BITS, int NT>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 4 : 3) stream_kernel(const AttnParams P) {
  using St = Stream<BITS, NT>;
  constexpr int R = St::R, RB = St::RB;
  __shared__ float sm_o[WARPS][R][D];
  __shared__ float sm_m[WARPS][R], sm_l[WARPS][R];
  __shared__ int64_t sm_scan[WARPS];
  __shared__ int64_t sm_total, sm_base;
  __shared__ int sm_b;
  __shared__ bool sm_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = P.G, hkv = P.pages.hkv, B = P.batch.B;
  const bool split = P.part != nullptr;

  // ---- the list: this CTA's piece, and the sequence it begins in
  auto weight = [&](const Seq& s, int& per) {
    const int nrt = s.qlen * G > P.many_rows ? 0 : (s.qlen * G + R - 1) / R;
    per = split ? max(s.tiles(), 1) : 1;   // tiles per unit; a unit without keys still writes zeros
    return static_cast<int64_t>(nrt) * hkv * per;
  };
  const int chunk = (B + THREADS - 1) / THREADS;
  int64_t mine = 0;
  for (int b = tid * chunk; b < min(B, (tid + 1) * chunk); ++b) {
    int per;
    mine += weight(load_seq(P, b, blockIdx.x == 0), per);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm_scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sm_scan[w];
    total += sm_scan[w];
  }
  const int64_t excl = before + incl - mine;
  // every CTA of the list holds a tile, so a unit's pieces belong to consecutive CTAs
  const int ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const int64_t r0 = total * blockIdx.x / ctas, r1 = total * (blockIdx.x + 1) / ctas;
  if (r0 >= excl && r0 < excl + mine) {
    int b = tid * chunk;
    int64_t base = excl;
    for (;; ++b) {
      int per;
      const int64_t w = weight(load_seq(P, b, false), per);
      if (r0 < base + w) break;
      base += w;
    }
    sm_b = b;
    sm_base = base;
  }
  __syncthreads();
  int b = sm_b;
  int64_t base = sm_base;

  for (int64_t cur = r0; cur < r1;) {
    Unit u;
    u.s = load_seq(P, b, false);
    int per;
    const int64_t wgt = weight(u.s, per);
    if (cur >= base + wgt) {
      base += wgt;
      ++b;
      continue;
    }
    const int64_t unit = (cur - base) / per;
    const int i0 = static_cast<int>((cur - base) - unit * per);
    const int i1 = static_cast<int>(min(static_cast<int64_t>(per), i0 + (r1 - cur)));
    const int64_t u0 = base + unit * per;  // the unit's place in the list
    const bool whole = i0 == 0 && i1 == per;
    u.b = b;
    u.h = static_cast<int>(unit % hkv);
    u.row0 = static_cast<int>(unit / hkv) * R;
    u.rows = min(R, u.s.qlen * G - u.row0);
    cur += i1 - i0;
    const int first = split ? i0 : 0, last = split ? min(i1, u.s.tiles()) : u.s.tiles();

    uint32_t qb[NT][8][2];
    float qf[NT][2];
    St::load_q(P, u, g, t, qb, qf);
    // this thread's columns: rows 8 n + 2 t + {0, 1}
    int qpos[NT][2];
    float slope[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = min(8 * n + 2 * t + e, u.rows - 1);
        const int tok = (u.row0 + r) / G;
        qpos[n][e] = u.s.pos0 + tok;
        slope[n][e] = P.slopes ? P.slopes[u.h * G + u.row0 + r - tok * G] * kLog2e : 0.f;
      }

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
    float svr = 0.f, svi = 0.f;            // power of two at or above the value scales so far; 1 / svr

    for (int i = first; i < last; ++i) {
      const bool pre = i < u.s.pn;
      const int local = (pre ? u.s.pt0 + i : u.s.ot0 + i - u.s.pn) * TILE + 16 * warp;
      const int limit = pre ? P.prefix_len : u.s.len;
      if (local >= limit) continue;
      const int kpos0 = (pre ? 0 : P.prefix_len) + local;      // position of the warp's first key
      const int32_t* table =
          pre ? P.prefix_table : P.batch.table + static_cast<int64_t>(u.b) * P.batch.width;
      const int page = table[local >> P.pages.lps];
      if (page < 0 || page >= P.pages.num_pages) {
        if (lane == 0) record_status(SQ_ERR_INVALID_ARG);
        continue;
      }
      const int64_t grp = group_of(P.pages, page, u.h, local & ((1 << P.pages.lps) - 1));
      // ---- loads
      KFrag<BITS> kf[2];
      VFrag<BITS> vf[4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint4* src = reinterpret_cast<const uint4*>(P.pages.kc + (grp + g + 8 * hf) * RB) + t;
#pragma unroll
        for (int c = 0; c < BITS / 4; ++c) kf[hf].c[c] = __ldg(src + 4 * c);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 2 * t + (j & 1) + 8 * (j >> 1);
        const uint2* src =
            reinterpret_cast<const uint2*>(P.pages.vc + (grp + key) * RB + g * (RB / 8));
#pragma unroll
        for (int c = 0; c < BITS / 4; ++c) vf[j].c[c] = __ldg(src + c);
      }
      float sk[2], sv[2];
      __half2 kz1[2], kz16[2], vz1[2], vz16[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        sk[hf] = __ldg(P.pages.ks + grp + g + 8 * hf);
        sv[hf] = __ldg(P.pages.vs + grp + g + 8 * hf);
        const int z = __ldg(P.pages.kz + grp + g + 8 * hf);
        kz1[hf] = __half2half2(__int2half_rn(-1024 - z));
        kz16[hf] = __half2half2(__int2half_rn(-64 - z));
        const uint32_t zz =
            __ldg(reinterpret_cast<const uint16_t*>(P.pages.vz + grp) + t + 4 * hf);
        const int za = zz & 0xFF, zb = zz >> 8;
        vz1[hf] = __halves2half2(__int2half_rn(-1024 - za), __int2half_rn(-1024 - zb));
        vz16[hf] = __halves2half2(__int2half_rn(-64 - za), __int2half_rn(-64 - zb));
      }
      // ---- S^T = K_int Q^T
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(kf[0].c);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(kf[1].c);
#pragma unroll
      for (int w = 0; w < BITS; ++w) {
        if (BITS == 4) {
          uint32_t x[4], y[4];
          widen_nibbles(w0[w], kz1[0], kz16[0], x);
          widen_nibbles(w1[w], kz1[1], kz16[1], y);
          const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(sc[n], a0, qb[n][2 * w][0], qb[n][2 * w][1]);
            mma16816(sc[n], a1, qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
          }
        } else {
          uint32_t x[2], y[2];
          widen_bytes(w0[w], kz1[0], x);
          widen_bytes(w1[w], kz1[1], y);
          const uint32_t a[4] = {x[0], y[0], x[1], y[1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(sc[n], a, qb[n][w][0], qb[n][w][1]);
        }
      }
      // ---- scores: [n][0], [1] key g; [2], [3] key g + 8; columns 2t, 2t + 1
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int hf = e >> 1, c = e & 1;
          float x = sc[n][e] * sk[hf] * qf[n][c];
          if (P.cap > 0.f) x = P.cap * kLog2e * tanh_score(x);
          const int dist = qpos[n][c] - (kpos0 + g + 8 * hf);
          x = fmaf(-slope[n][c], static_cast<float>(dist), x);
          const bool seen =
              dist >= 0 && (P.window == 0 || dist < P.window) && local + g + 8 * hf < limit;
          sc[n][e] = seen ? x : -INFINITY;
          raise |= sc[n][e] > m[n][c] + (kLift + kLazy);
        }
      // ---- references: rescale only when a maximum has moved far
      float svmax = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {     // infinities and NaN, and rows behind the last key, set none
        const float a = fabsf(sv[hf]);
        svmax = fmaxf(svmax, local + g + 8 * hf < limit && a <= 3.0e38f ? a : 0.f);
      }
      raise |= svmax > svr;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int of = 4; of < 32; of <<= 1)
          svmax = fmaxf(svmax, __shfl_xor_sync(0xffffffffu, svmax, of));
        // a power of two at or above svmax, between 2^-126 and 2^126
        const int e2 = max(1, min(253, static_cast<int>(__float_as_uint(svmax) >> 23) + 1));
        const float nsv = fmaxf(svr, __uint_as_float(static_cast<uint32_t>(e2) << 23));
        const float down = svr > 0.f ? svr / nsv : 0.f;
        svr = nsv;
        svi = 1.0f / nsv;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(sc[n][c], sc[n][2 + c]) - kLift, m[n][c]);
#pragma unroll
            for (int of = 4; of < 32; of <<= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, of));
            const float f = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - mx);
            m[n][c] = mx;
            l[n][c] *= f;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[n][i8][c] *= f * down;
              o[n][i8][2 + c] *= f * down;
            }
          }
      }
      // ---- weights, as fp16 pairs (high, low), to the B operand's layout
      uint32_t ph[NT][2], pl[NT][2];
      const float wv[2] = {sv[0] * svi, sv[1] * svi};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float w[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = sc[n][2 * hf + c];
            const float p = x == -INFINITY ? 0.f : ex2(x - m[n][c]);
            l[n][c] += p;
            w[c] = p == 0.f ? 0.f : p * wv[hf];
          }
          const __half2 hi = __floats2half2_rn(w[0], w[1]);
          const float2 back = __half22float2(hi);
          ph[n][hf] = transpose8x8(h2_bits(hi));
          pl[n][hf] = transpose8x8(h2_bits(__floats2half2_rn(w[0] - back.x, w[1] - back.y)));
        }
      // ---- O^T += V_int^T w: dims 16 g + 2 i + {0, 1} in m-tile i
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t va[8], vb[8];             // 8 dims of key pairs (2t, 2t+1) and (2t+8, 2t+9)
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          uint32_t(&dst)[8] = pr ? vb : va;
          if (BITS == 4) {
            const uint32_t a = half ? vf[2 * pr].c[0].y : vf[2 * pr].c[0].x;
            const uint32_t bb = half ? vf[2 * pr + 1].c[0].y : vf[2 * pr + 1].c[0].x;
            uint32_t x[4];
#pragma unroll
            for (int hw = 0; hw < 2; ++hw) {
              const uint32_t mix = __byte_perm(a, bb, hw ? 0x7632u : 0x5410u);
              const __half2 six = __float2half2_rn(0.0625f);
              const uint32_t m8 = mix >> 8;
              x[0] = h2_bits(__hadd2(bits_h2((mix & 0x000F000Fu) | 0x64006400u), vz1[pr]));
              x[1] = h2_bits(__hfma2(bits_h2((mix & 0x00F000F0u) | 0x64006400u), six, vz16[pr]));
              x[2] = h2_bits(__hadd2(bits_h2((m8 & 0x000F000Fu) | 0x64006400u), vz1[pr]));
              x[3] = h2_bits(__hfma2(bits_h2((m8 & 0x00F000F0u) | 0x64006400u), six, vz16[pr]));
#pragma unroll
              for (int e = 0; e < 4; ++e) dst[4 * hw + e] = x[e];
            }
          } else {
            const uint2 a2 = vf[2 * pr].c[BITS == 4 ? 0 : half];
            const uint2 b2 = vf[2 * pr + 1].c[BITS == 4 ? 0 : half];
#pragma unroll
            for (int hw = 0; hw < 2; ++hw) {
              const uint32_t a = hw ? a2.y : a2.x, bb = hw ? b2.y : b2.x;
              const uint32_t lo = __byte_perm(a, bb, 0x5140u), hi = __byte_perm(a, bb, 0x7362u);
              uint32_t x[2], y[2];
              widen_bytes(lo, vz1[pr], x);
              widen_bytes(hi, vz1[pr], y);
              dst[4 * hw] = x[0], dst[4 * hw + 1] = x[1];
              dst[4 * hw + 2] = y[0], dst[4 * hw + 3] = y[1];
            }
          }
        }
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const uint32_t a[4] = {va[2 * i4], va[2 * i4 + 1], vb[2 * i4], vb[2 * i4 + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(o[n][4 * half + i4], a, ph[n][0], ph[n][1]);
            mma16816(o[n][4 * half + i4], a, pl[n][0], pl[n][1]);
          }
        }
      }
    }

    // ---- the warps' results into shared memory, at a common maximum
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], of);
        if (g == 0) {
          sm_m[warp][8 * n + 2 * t + c] = m[n][c];
          sm_l[warp][8 * n + 2 * t + c] = l[n][c];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float2*>(&sm_o[warp][8 * n + 2 * t + c][16 * g + 2 * i]) =
              make_float2(o[n][i][c] * svr, o[n][i][2 + c] * svr);
      }
    __syncthreads();
    // thread tid owns dim tid of every row
    const int64_t c0 = ((u0 + 1) * ctas - 1) / total;            // CTA that holds the unit's first tile
    const int64_t c1 = ((u0 + per) * ctas - 1) / total;          // and its last
    const int slot = 2 * blockIdx.x + (u0 >= r0 ? 1 : 0);
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
        if (f != 0.f) acc[r] = fmaf(f, sm_o[w][r][tid], acc[r]);
        ll[r] = fmaf(f, sm_l[w][r], ll[r]);
      }
    }
    bool finish = whole;
    if (!whole) {
      float* p = P.part + static_cast<int64_t>(slot) * PART;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        p[r * D + tid] = acc[r];
        if (tid == 0) {
          p[R * D + r] = mm[r];
          p[R * D + R + r] = ll[r];
        }
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
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
        for (int64_t c = c0; c <= c1; ++c) {
          const int64_t cb = total * c / ctas;
          const float* p2 = P.part + (2 * c + (u0 >= cb ? 1 : 0)) * PART;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float pm = __ldcg(p2 + R * D + r), plv = __ldcg(p2 + R * D + R + r);
            const float M = fmaxf(mm[r], pm);
            const float fa = mm[r] == -INFINITY ? 0.f : ex2(mm[r] - M);
            const float fb = pm == -INFINITY ? 0.f : ex2(pm - M);
            const float po = __ldcg(p2 + r * D + tid);
            acc[r] = fa * acc[r] + (fb != 0.f ? fb * po : 0.f);
            ll[r] = fa * ll[r] + fb * plv;
            mm[r] = M;
          }
        }
      }
    }
    if (finish) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r < u.rows) {
          const int tok = (u.row0 + r) / G, head = u.h * G + u.row0 + r - tok * G;
          const int64_t row = static_cast<int64_t>(u.s.row0 + tok) * P.hq + head;
          // the shared prefix's part of the row, in pieces
          for (int e = 0; e < P.ex_n; ++e) {
            const int64_t at = static_cast<int64_t>(e) * P.batch.T * P.hq + row;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(P.ex_ml) + at);
            const float po = __ldcg(P.ex_o + at * D + tid);
            const float M = fmaxf(mm[r], ml.x);
            const float fa = mm[r] == -INFINITY ? 0.f : ex2(mm[r] - M);
            const float fb = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            acc[r] = fa * acc[r] + (fb != 0.f ? fb * po : 0.f);
            ll[r] = fa * ll[r] + fb * ml.y;
            mm[r] = M;
          }
          const float y = ll[r] == 0.f ? 0.f : acc[r] / ll[r];
          P.out[row * D + tid] = __float2bfloat16_rn(y);
          if (P.lse && tid == r) P.lse[row] = ll[r] == 0.f ? -INFINITY : (mm[r] + log2f(ll[r])) * kLn2;
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

template <int BITS, int NT>
int grid_size() {
  static int cache[64] = {0};
  const int d = host::current_device();
  if (d >= 0 && d < 64 && cache[d] > 0) return cache[d];
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, stream_kernel<BITS, NT>, THREADS, 0) !=
          cudaSuccess ||
      per_sm < 1) {
    (void)cudaGetLastError();
    per_sm = 1;
  }
  const int grid = host::num_sms() * per_sm < kMaxGrid ? host::num_sms() * per_sm : kMaxGrid;
  if (d >= 0 && d < 64) cache[d] = grid;
  return grid;
}

int any_grid(int bits, int nt) {
  if (bits == 4) return nt == 1 ? grid_size<4, 1>() : grid_size<4, 2>();
  return nt == 1 ? grid_size<8, 1>() : grid_size<8, 2>();
}

// Sequences of up to this many rows (new tokens x query heads per KV head)
// go to the streaming kernel, longer ones to the tile kernel.
constexpr int kFewRows = 16;
// A shared prefix is read once for the batch while no sequence has more rows
// than this; longer ones fill the tile kernel's rows by themselves.
constexpr int kSharedRows = 128;
constexpr int kTileRows = 256;
constexpr size_t kPartFloats = static_cast<size_t>(kTileRows) * (D + 2);

AttnPlan make_plan(int64_t T, int hq, int hkv, int B, int max_q, int64_t keys, int prefix_len,
                   int bits, bool have_ws) {
  AttnPlan p{};
  const int64_t G = hq / hkv, rows = G * max_q;
  const int sms = host::num_sms();
  p.nt = rows <= 8 ? 1 : 2;
  p.shared = prefix_len > 0 && rows <= kSharedRows && B > 1 && have_ws;
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
    p.part = take(static_cast<size_t>(any_grid(bits, p.nt)) * 2 * (8 * p.nt) * (D + 2) * 4);
  if (p.shared) {
    const int64_t units = (T * G + kTileRows - 1) / kTileRows * hkv, tiles = (prefix_len + 127) / 128;
    int64_t s = sms / units;
    if (s > (tiles + 1) / 2) s = (tiles + 1) / 2;
    p.tile_split = static_cast<int>(s < 1 ? 1 : s);
    p.tile_units = units * p.tile_split;
    p.ex_o = take(static_cast<size_t>(p.tile_split) * T * hq * D * 4);
    p.ex_ml = take(static_cast<size_t>(p.tile_split) * T * hq * 2 * 4);
  } else if (p.tile) {
    const int64_t slots = (T * G / kTileRows + B) * hkv, tiles = (keys + prefix_len + 127) / 128;
    int64_t s = have_ws ? 2 * sms / slots : 1;
    if (s > (tiles + 1) / 2) s = (tiles + 1) / 2;
    if (s < 1 || slots > static_cast<int64_t>(kCountBytes / 4)) s = 1;
    p.tile_split = static_cast<int>(s);
    p.tile_units = slots * s;
    if (s > 1) p.tpart = take(static_cast<size_t>(slots) * s * kPartFloats * 4);
  }
  p.bytes = at;
  return p;
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int hq, int hkv, int B, int max_q, int64_t keys,
                                 int prefix_len, int bits) {
  return make_plan(T, hq, hkv, B, max_q, keys, prefix_len, bits, true).bytes;
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
  P.window = rule.window;
  P.slopes = rule.slopes;
  P.out = static_cast<__nv_bfloat16*>(out);
  P.lse = lse;
  P.spin_limit = host::spin_limit();
  const int64_t keys = static_cast<int64_t>(width) * pages.page_size;
  AttnPlan plan = make_plan(T, hq, pages.hkv, B, max_q, keys, prefix_len, pages.bits, true);
  const bool have = ws && ws_bytes >= plan.bytes;
  if (!have) plan = make_plan(T, hq, pages.hkv, B, max_q, keys, prefix_len, pages.bits, false);
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
  if (plan.tile || plan.shared) {
    const sq_status st = launch_tile(P, pages.bits, stream);
    if (st != SQ_OK) return st;
  }
  if (!plan.stream) return SQ_OK;
  P.ex_n = plan.shared ? plan.tile_split : 0;
  const int grid = any_grid(pages.bits, plan.nt);
  auto kern = pages.bits == 4 ? (plan.nt == 1 ? stream_kernel<4, 1> : stream_kernel<4, 2>)
                              : (plan.nt == 1 ? stream_kernel<8, 1> : stream_kernel<8, 2>);
  kern<<<grid, THREADS, 0, stream>>>(P);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv attention launch", e);
}

}  // namespace paged
}  // namespace sq
