// The paged 4/8-bit KV cache, sm_100a: appending a ragged batch's new tokens
// (per-head RMS norm, rotary embedding, R3, asymmetric quantization) and
// reading rows back.
//
// One head vector of 128 values per 8 lanes: lane s holds the 16-byte chunks
// s and s + 8 (elements 8 s + e and 64 + 8 s + e), so a warp loads four whole
// vectors with two instructions of full sectors.  All the maps are linear
// but the norm's factor, which is one number per vector, so
//     y = f * H (R (w * x)),  f = rsqrt(mean x^2 + eps) / sqrt(128)
// with R the rotary map: the factor is applied once, after the butterflies.
// The usual rotary map (half layout, whole head) pairs a lane's two chunks, so
// its cosines and sines stay in registers for all of a token's heads; for the
// others (interleaved, or part of the head, any multiple of 16) the partner's
// chunk is read again (an L1 hit) rather than exchanged between lanes.
// H128's bits 0-2 and 6 run inside the lane, bits 3-5 across the 8 lanes.
//
// A warp takes a token (or, for few tokens, a part of its heads): it finds the
// token's place once, while the first heads' values are already on their way,
// and always has the next heads' loads in flight.
//
// What bounds it: issue slots (70 %) and the shuffles of the cross-lane stages;
// 16,384 tokens of 32 + 2 x 8 heads at 4 bits take 114 us (354 MB, 54 us of
// HBM; 112 before queries of any size were taken) and their read-back 23 right
// behind it, 29 from cold caches (85 MB, 13; bound by the chain from a token to
// its rows), both together 270 with a warp per job that looked its token up again
// and waited for its loads.  Registers for 3 CTAs an SM: of an earlier form that
// took 113 us, 2 took 120, 4 (spills) 138.
//
// Q is computed in float32 (its output is bf16).  K is computed in double
// precision and rounded once to float32, so its codes are those of the exact
// rotation (the contiguous cache's rule); V is quantized as it is.
#include <cuda_bf16.h>
#include <math.h>

#include "kv_paged.cuh"
#include "kv_quant.cuh"
#include "sq_device.cuh"
#include "sq_host.h"

namespace sq {
namespace paged {

constexpr int LPV = 8;                     // lanes per head vector
constexpr int VPW = 32 / LPV;              // head vectors per warp

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  int64_t sq, sk, sv;                      // elements between tokens
  Pages pages;
  Batch batch;
  const float *cos, *sin;                  // [max_pos][rot / 2], or null
  int max_pos, rot, interleaved;
  const float *q_norm, *k_norm;            // [128], or null
  float eps;
  __nv_bfloat16* q_out;
  int hq, jq, jk;                          // query heads; warp jobs per token of Q and of K
  int split;                               // warps per token
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(ws[e] << 16);
    x[2 * e + 1] = __uint_as_float(ws[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void chunk8(const __nv_bfloat16* p, float (&x)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), x);
}

__device__ __forceinline__ void floats8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The rotary factors of a token that a lane keeps (half layout, whole head:
// pairs 8 s .. 8 s + 7, channel 8 s + e with 64 + 8 s + e).
struct Factors {
  float c[8], s[8];
};

// y = H128's bits 3-5, across the 8 lanes of a vector.
template <class R>
__device__ __forceinline__ void across(R (&y)[16], int s, unsigned mask) {
#pragma unroll
  for (int o = 1; o < LPV; o <<= 1) {
    const R sg = (s & o) ? R(-1) : R(1);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = fma(sg, y[e], __shfl_xor_sync(mask, y[e], o));
  }
}

// R (w * x) of one vector over its 8 lanes, in R's precision, and the norm's
// sum of squares of this lane's values.  raw: chunks s and s + 8.
template <class R, bool WHOLE>
__device__ __forceinline__ R scale_and_turn(const uint4 (&raw)[2], const __nv_bfloat16* src, const float* w,
                                            const Factors& fac, const float* cs, const float* sn,
                                            int rot, bool interleaved, int s, R (&y)[16], float scale = 1.0f) {
  R sum = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float x[8], g[8];
    unpack8(raw[c], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[8 * c + e] = x[e];
    if (w) {
      floats8(w + 64 * c + 8 * s, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += static_cast<R>(x[e]) * static_cast<R>(x[e]);
        y[8 * c + e] *= static_cast<R>(g[e]);
      }
    }
  }
  if (WHOLE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const R a = y[e], b = y[8 + e], C = fac.c[e], S = fac.s[e];
      y[e] = a * C - b * S;
      y[8 + e] = b * C + a * S;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = 64 * c + 8 * s;
    if (WHOLE || e0 >= rot) continue;
    if (interleaved) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + e0 / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(sn + e0 / 2));
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const R a = y[8 * c + 2 * e], b = y[8 * c + 2 * e + 1];
        const R C = cc[e], S = ss[e];
        y[8 * c + 2 * e] = a * C - b * S;
        y[8 * c + 2 * e + 1] = b * C + a * S;
      }
    } else {
      const int half = rot >> 1;
      const bool upper = e0 >= half;
      const int p0 = upper ? e0 - half : e0 + half, i0 = upper ? p0 : e0;
      float b[8], cc[8], ss[8], g[8];
      chunk8(src + p0, b);
      floats8(cs + i0, cc);
      floats8(sn + i0, ss);
      if (w) floats8(w + p0, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        R t = sizeof(R) == 4 ? b[e] * scale : b[e];        // (the lane's own values have it already)
        if (w) t *= static_cast<R>(g[e]);
        t *= static_cast<R>(ss[e]);
        y[8 * c + e] = y[8 * c + e] * static_cast<R>(cc[e]) + (upper ? t : -t);
      }
    }
  }
  return sum;
}

// A query whose squares float32 does not hold (values past 1e18, or all below 1e-15 with an eps as small) is
// taken again by this or its reciprocal: the norm does not depend on it.
constexpr float kUp = 1.2089258e24f;       // 2^80

// f H, f = rsqrt(mean x^2 + eps) / sqrt(128) (w) or 1 / sqrt(128): in double.
__device__ __forceinline__ void finish(double (&y)[16], double sum, bool norm, float eps, int s, unsigned mask) {
  double f = 0.088388347648318440550;      // 1/sqrt(128)
  if (norm) {
#pragma unroll
    for (int o = 1; o < LPV; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
    f *= 1.0 / sqrt(sum * (1.0 / D) + static_cast<double>(eps));
  }
#pragma unroll
  for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if ((e & h) == 0) {
        const double a = y[e], b = y[e + h];
        y[e] = a + b;
        y[e + h] = a - b;
      }
    }
  }
  across(y, s, mask);
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] *= f;
}

// The same in float32, two values (the lane's two chunks) an instruction, of a vector of `scale` times its
// values.  False where its mean square leaves float32: then `scale` is the power of two to take it by.
__device__ __forceinline__ bool finish(float (&y)[16], float sum, bool norm, float eps, int s, unsigned mask,
                                       float& scale) {
  float f = 0.088388347648318440550f;
  if (norm) {
#pragma unroll
    for (int o = 1; o < LPV; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
    const float mean = sum * (1.0f / D) + eps * scale * scale;
    if (scale == 1.0f && !(mean >= 1e-30f && mean <= 1e34f)) {
      scale = mean < 1.0f ? kUp : 1.0f / kUp;
      return false;
    }
    f *= 1.0f / sqrtf(mean);
  }
  f2 v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = f2{(y[e] + y[8 + e]) * f, (y[e] - y[8 + e]) * f};
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((e & h) == 0) {
        const f2 a = v[e], b = v[e + h];
        v[e] = add2(a, b);
        v[e + h] = sub2(a, b);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < LPV; o <<= 1) {
    const float sg = (s & o) ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = fma2(f2{sg, sg}, v[e],
                  f2{__shfl_xor_sync(mask, v[e].x, o), __shfl_xor_sync(mask, v[e].y, o)});
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = v[e].x, y[8 + e] = v[e].y;
  return true;
}

// Quantizes one vector held by 8 lanes (lane s: chunks s and s + 8) into row
// `g` of a cache.
template <int BITS>
__device__ __forceinline__ void store_quantized(const float (&y)[16], int s, unsigned mask,
                                                uint8_t* codes, float* scales, uint8_t* zeros,
                                                int64_t g) {
  float mn = y[0], mx = y[0];
#pragma unroll
  for (int e = 1; e < 16; ++e) {
    mn = fminf(mn, y[e]);
    mx = fmaxf(mx, y[e]);
  }
  float scale, zero;
  kv::asym_params<BITS, LPV>(mn, mx, mask, scale, zero);
  // scale and inputs times 2^64 when the scale is subnormal (see ucodes8_div)
  const float up = scale < 1.17549435e-38f ? 18446744073709551616.0f : 1.0f;
  const float su = scale * up;
  const float rs = __frcp_rn(su);
  const f2 u2{up, up}, r2{rs, rs}, sn2{-su, -su}, z2{zero, zero};
  constexpr int RB = D * BITS / 8;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float* v = y + 8 * c;
    const f2 xs[4] = {f2{v[0], v[1]}, f2{v[2], v[3]}, f2{v[4], v[5]}, f2{v[6], v[7]}};
    uint32_t w[BITS / 4];
    kv::ucodes8_div<BITS>(xs, u2, r2, sn2, z2, w);
    uint8_t* dst = codes + g * RB + (s + LPV * c) * BITS;
    if (BITS == 4)
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[BITS / 4 - 1]);
  }
  if (s == 0) {
    scales[g] = scale;
    zeros[g] = static_cast<uint8_t>(zero);
  }
}

// WHOLE: half layout over the whole head.
template <int BITS, bool WHOLE>
__global__ void __launch_bounds__(256, 3) append_kernel(const AppendParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, s = lane & (LPV - 1), vec = lane / LPV;
  const unsigned mask = 0xFFu << (lane & 24);
  const int jobs = P.jq + 2 * P.jk;        // four heads each: Q, K, V
  const int64_t items = P.batch.T * P.split;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int64_t t = P.split == 1 ? it : it / P.split;
    const int part = static_cast<int>(it - t * P.split);
    // this lane's head of a job, the last one where there are no four (what it gives is not stored)
    auto source = [&](int job) {
      if (job < P.jq) return P.q + t * P.sq + min(job * VPW + vec, P.hq - 1) * D;
      job -= P.jq;
      const bool is_v = job >= P.jk;
      const int head = min((is_v ? job - P.jk : job) * VPW + vec, P.pages.hkv - 1);
      return is_v ? P.v + t * P.sv + head * D : P.k + t * P.sk + head * D;
    };
    const __nv_bfloat16* src = source(part);
    uint4 raw[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) raw[c] = *reinterpret_cast<const uint4*>(src + 64 * c + 8 * s);
    int pos, page;
    bool bad;
    bool ok = locate(P.pages, P.batch, t, pos, page, bad);
    if (ok && P.cos && pos >= P.max_pos) bad = true, ok = false;
    if (!ok) {
      if (bad && lane == 0 && part == 0) record_status(SQ_ERR_INVALID_ARG);
      continue;
    }
    const float* cs = P.cos + static_cast<int64_t>(pos) * (P.rot >> 1);
    const float* sn = P.sin + static_cast<int64_t>(pos) * (P.rot >> 1);
    Factors fac;
    if (WHOLE) {
      floats8(cs + 8 * s, fac.c);
      floats8(sn + 8 * s, fac.s);
    }
    for (int job = part; job < jobs; job += P.split) {
      const __nv_bfloat16* now = src;
      const uint4 mine[2] = {raw[0], raw[1]};
      if (job + P.split < jobs) {
        src = source(job + P.split);
#pragma unroll
        for (int c = 0; c < 2; ++c) raw[c] = *reinterpret_cast<const uint4*>(src + 64 * c + 8 * s);
      }
      if (job < P.jq) {
        const int head = job * VPW + vec;
        float y[16], scale = 1.0f;
        uint4 in[2] = {mine[0], mine[1]};
#pragma unroll 1
        for (;;) {
          const float sum = scale_and_turn<float, WHOLE>(in, now, P.q_norm, fac, cs, sn, P.rot, P.interleaved, s, y, scale);
          if (finish(y, sum, P.q_norm != nullptr, P.eps, s, mask, scale)) break;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            in[c] = *reinterpret_cast<const uint4*>(now + 64 * c + 8 * s);
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&in[c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], __float2bfloat162_rn(scale));
          }
        }
        if (head < P.hq) {
          __nv_bfloat16* dst = P.q_out + (t * P.hq + head) * D + 8 * s;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float* v = y + 8 * c;
            *reinterpret_cast<uint4*>(dst + 64 * c) =
                make_uint4(kv::bf16x2(v[0], v[1]), kv::bf16x2(v[2], v[3]), kv::bf16x2(v[4], v[5]),
                           kv::bf16x2(v[6], v[7]));
          }
        }
        continue;
      }
      const bool is_v = job >= P.jq + P.jk;
      const int head = (job - P.jq - (is_v ? P.jk : 0)) * VPW + vec;
      float x[16];
      if (is_v) {
        float a[8], b[8];
        unpack8(mine[0], a);
        unpack8(mine[1], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = a[e], x[8 + e] = b[e];
      } else {
        double y[16];
        const double sum = scale_and_turn<double, WHOLE>(mine, now, P.k_norm, fac, cs, sn, P.rot, P.interleaved, s, y);
        finish(y, sum, P.k_norm != nullptr, P.eps, s, mask);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = static_cast<float>(y[e]);
      }
      if (head < P.pages.hkv) {            // whole groups of 8 lanes
        const int64_t g = group_of(P.pages, page, head, pos & ((1 << P.pages.lps) - 1));
        store_quantized<BITS>(x, s, mask, is_v ? P.pages.vc : P.pages.kc, is_v ? P.pages.vs : P.pages.ks,
                              is_v ? P.pages.vz : P.pages.kz, g);
      }
    }
  }
}

// Rows of the pages back to bf16, 16 lanes per head vector (8 codes each).
template <int BITS>
__global__ void __launch_bounds__(256) dequant_kernel(const Pages P, const Batch b, __nv_bfloat16* k_out,
                                                      __nv_bfloat16* v_out, int split) {
  constexpr int RB = D * BITS / 8;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, c = lane & 15;
  const bool is_v = lane >= 16;            // a job: one head's K and V
  const uint8_t* codes = is_v ? P.vc : P.kc;
  const float* scales = is_v ? P.vs : P.ks;
  const uint8_t* zeros = is_v ? P.vz : P.kz;
  __nv_bfloat16* out = is_v ? v_out : k_out;
  const int64_t items = b.T * split;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items;
       it += step) {
    const int64_t t = split == 1 ? it : it / split;
    const int part = static_cast<int>(it - t * split);
    int pos, page;
    bool bad;
    if (!locate(P, b, t, pos, page, bad)) {
      if (bad && part == 0 && lane == 0) record_status(SQ_ERR_INVALID_ARG);
      continue;
    }
    const int64_t g0 = group_of(P, page, 0, pos & ((1 << P.lps) - 1));
#pragma unroll 4
    for (int head = part; head < P.hkv; head += split) {
      const int64_t g = g0 + (static_cast<int64_t>(head) << P.lps);
      const uint8_t* src = codes + g * RB + c * BITS;
      const float scale = __ldg(scales + g);
      const float zb = 8388608.0f + static_cast<float>(__ldg(zeros + g));
      uint2 w;
      if (BITS == 4)
        w = make_uint2(__ldg(reinterpret_cast<const uint32_t*>(src)), 0u);
      else
        w = __ldg(reinterpret_cast<const uint2*>(src));
      *reinterpret_cast<uint4*>(out + (t * P.hkv + head) * D + 8 * c) = kv::widen8<BITS>(w, scale, zb);
    }
  }
}

namespace {

Pages view(const sq_kv_pages& p) {
  Pages v{p.k_codes, p.k_scale, p.k_zero, p.v_codes, p.v_scale, p.v_zero, p.num_pages, 0, p.hkv};
  while ((1 << v.lps) < p.page_size) ++v.lps;
  return v;
}

// Warps per token: one while that fills the device (32 warps per SM), else as many as it takes, a
// job each at most.
int warps_per_token(int64_t T, int jobs) {
  const int64_t want = (static_cast<int64_t>(host::num_sms()) * 32 + T - 1) / T;
  return static_cast<int>(want < jobs ? want : jobs);
}

int grid_for(int64_t warps, int per_sm) {
  const int64_t want = (warps + 7) / 8, cap = static_cast<int64_t>(host::num_sms()) * per_sm;
  return static_cast<int>(want < cap ? want : cap);
}

}  // namespace

sq_status run_append(const void* q, const void* k, const void* v, int64_t q_stride,
                     int64_t k_stride, int64_t v_stride, int64_t T, int hq,
                     const sq_kv_pages& pages, const int32_t* table, int width, const int32_t* cu,
                     const int32_t* cached, int B, const float* cos, const float* sin, int max_pos,
                     int rot, int interleaved, const float* q_norm, const float* k_norm, float eps,
                     void* q_out, cudaStream_t stream) {
  AppendParams P;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.k = static_cast<const __nv_bfloat16*>(k);
  P.v = static_cast<const __nv_bfloat16*>(v);
  P.sq = q_stride, P.sk = k_stride, P.sv = v_stride;
  P.pages = view(pages);
  P.batch = Batch{table, cu, cached, width, B, T};
  P.cos = cos, P.sin = sin;
  P.max_pos = max_pos, P.rot = cos ? rot : 0, P.interleaved = interleaved;
  P.q_norm = q_norm, P.k_norm = k_norm, P.eps = eps;
  P.q_out = static_cast<__nv_bfloat16*>(q_out);
  P.hq = hq;
  P.jq = (hq + VPW - 1) / VPW;
  P.jk = (pages.hkv + VPW - 1) / VPW;
  P.split = warps_per_token(T, P.jq + 2 * P.jk);
  const bool whole = cos && rot == D && !interleaved;
  auto kern = pages.bits == 8 ? (whole ? append_kernel<8, true> : append_kernel<8, false>)
                              : (whole ? append_kernel<4, true> : append_kernel<4, false>);
  const cudaError_t e =
      host::launch_dependent(kern, grid_for(T * P.split, 8), 256, 0, stream, P);
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv_paged_append launch", e);
}

sq_status run_dequant(const sq_kv_pages& pages, const int32_t* table, int width, const int32_t* cu,
                      const int32_t* cached, int B, int64_t T, void* k_out, void* v_out,
                      cudaStream_t stream) {
  auto kern = pages.bits == 8 ? dequant_kernel<8> : dequant_kernel<4>;
  const int split = warps_per_token(T, pages.hkv);
  const cudaError_t e = host::launch_dependent(
      kern, grid_for(T * split, 8), 256, 0, stream, view(pages),
      Batch{table, cu, cached, width, B, T}, static_cast<__nv_bfloat16*>(k_out),
      static_cast<__nv_bfloat16*>(v_out), split);
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv_paged_dequant launch", e);
}

}  // namespace paged
}  // namespace sq
