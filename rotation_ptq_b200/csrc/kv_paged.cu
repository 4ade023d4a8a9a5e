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
// A rotary partner in the half layout sits rot / 2 channels away; its chunk is
// read again (an L1 hit) rather than exchanged between lanes, which serves
// every rot that is a multiple of 16 and both layouts with one data layout.
// H128's bits 0-2 and 6 run inside the lane, bits 3-5 across the 8 lanes.
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
};

__device__ __forceinline__ void chunk8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(ws[e] << 16);
    x[2 * e + 1] = __uint_as_float(ws[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void floats8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// y = f * H (R (w * x)) of one vector over its 8 lanes, in R's precision.
template <class R>
__device__ __forceinline__ void head_forward(const __nv_bfloat16* src, const float* w,
                                             const float* cs, const float* sn, int rot,
                                             bool interleaved, float eps, int s, unsigned mask,
                                             R (&y)[16]) {
  R sum = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = 64 * c + 8 * s;
    float x[8], g[8];
    chunk8(src + e0, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[8 * c + e] = x[e];
    if (w) {
      floats8(w + e0, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += static_cast<R>(x[e]) * static_cast<R>(x[e]);
        y[8 * c + e] *= static_cast<R>(g[e]);
      }
    }
    if (e0 < rot) {
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
        float b[8], cc[8], ss[8];
        chunk8(src + p0, b);
        floats8(cs + i0, cc);
        floats8(sn + i0, ss);
        if (w) floats8(w + p0, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          R t = b[e];
          if (w) t *= static_cast<R>(g[e]);
          t *= static_cast<R>(ss[e]);
          y[8 * c + e] = y[8 * c + e] * static_cast<R>(cc[e]) + (upper ? t : -t);
        }
      }
    }
  }
  R f = static_cast<R>(0.088388347648318440550);   // 1/sqrt(128)
  if (w) {
#pragma unroll
    for (int o = 1; o < LPV; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
    f *= R(1) / sqrt(sum * R(1.0 / D) + static_cast<R>(eps));
  }
#pragma unroll
  for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if ((e & h) == 0) {
        const R a = y[e], b = y[e + h];
        y[e] = a + b;
        y[e + h] = a - b;
      }
    }
  }
#pragma unroll
  for (int o = 1; o < LPV; o <<= 1) {
    const R sg = (s & o) ? R(-1) : R(1);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = fma(sg, y[e], __shfl_xor_sync(mask, y[e], o));
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] *= f;
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

template <int BITS>
__global__ void __launch_bounds__(256) append_kernel(AppendParams P) {
  const int lane = threadIdx.x & 31, s = lane & (LPV - 1), vec = lane / LPV;
  const unsigned mask = 0xFFu << (lane & 24);
  const int jobs = P.jq + 2 * P.jk;
  const int64_t n = P.batch.T * jobs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); j < n;
       j += step) {
    const int64_t t = j / jobs;
    int job = static_cast<int>(j - t * jobs);
    int pos, page;
    bool bad;
    bool ok = locate(P.pages, P.batch, t, pos, page, bad);
    if (ok && P.cos && pos >= P.max_pos) bad = true, ok = false;
    if (!ok) {
      if (bad && lane == 0 && job == 0) record_status(SQ_ERR_INVALID_ARG);
      continue;
    }
    const float* cs = P.cos + static_cast<int64_t>(pos) * (P.rot >> 1);
    const float* sn = P.sin + static_cast<int64_t>(pos) * (P.rot >> 1);
    if (job < P.jq) {
      const int head = job * VPW + vec;
      if (head >= P.hq) continue;          // whole groups of 8 lanes leave
      float y[16];
      head_forward<float>(P.q + t * P.sq + head * D, P.q_norm, cs, sn, P.rot, P.interleaved, P.eps,
                          s, mask, y);
      __nv_bfloat16* dst = P.q_out + (t * P.hq + head) * D + 8 * s;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float* v = y + 8 * c;
        *reinterpret_cast<uint4*>(dst + 64 * c) =
            make_uint4(kv::bf16x2(v[0], v[1]), kv::bf16x2(v[2], v[3]), kv::bf16x2(v[4], v[5]),
                       kv::bf16x2(v[6], v[7]));
      }
      continue;
    }
    job -= P.jq;
    const bool is_v = job >= P.jk;
    const int head = (is_v ? job - P.jk : job) * VPW + vec;
    if (head >= P.pages.hkv) continue;
    const int64_t g = group_of(P.pages, page, head, pos & ((1 << P.pages.lps) - 1));
    float x[16];
    if (is_v) {
      const __nv_bfloat16* src = P.v + t * P.sv + head * D + 8 * s;
      float a[8], b[8];
      chunk8(src, a);
      chunk8(src + 64, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = a[e], x[8 + e] = b[e];
      store_quantized<BITS>(x, s, mask, P.pages.vc, P.pages.vs, P.pages.vz, g);
    } else {
      double y[16];
      head_forward<double>(P.k + t * P.sk + head * D, P.k_norm, cs, sn, P.rot, P.interleaved, P.eps,
                           s, mask, y);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = static_cast<float>(y[e]);
      store_quantized<BITS>(x, s, mask, P.pages.kc, P.pages.ks, P.pages.kz, g);
    }
  }
}

// Rows of the pages back to bf16, 16 lanes per head vector (8 codes each).
template <int BITS>
__global__ void __launch_bounds__(256) dequant_kernel(Pages P, Batch b, __nv_bfloat16* k_out,
                                                      __nv_bfloat16* v_out) {
  constexpr int RB = D * BITS / 8;
  const int lane = threadIdx.x & 31, c = lane & 15;
  const int vecs = 2 * P.hkv;              // K heads, then V heads
  const int64_t n = b.T * P.hkv;           // warps take two vectors
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); j < n;
       j += step) {
    const int64_t t = j / P.hkv;
    const int vec = 2 * static_cast<int>(j - t * P.hkv) + (lane >> 4);
    int pos, page;
    bool bad;
    if (!locate(P, b, t, pos, page, bad)) {
      if (bad && vec == 0 && c == 0) record_status(SQ_ERR_INVALID_ARG);
      continue;
    }
    if (vec >= vecs) continue;
    const bool is_v = vec >= P.hkv;
    const int head = is_v ? vec - P.hkv : vec;
    const int64_t g = group_of(P, page, head, pos & ((1 << P.lps) - 1));
    const uint8_t* src = (is_v ? P.vc : P.kc) + g * RB + c * BITS;
    const float scale = (is_v ? P.vs : P.ks)[g];
    const float zb = 8388608.0f + static_cast<float>((is_v ? P.vz : P.kz)[g]);
    uint2 w;
    if (BITS == 4)
      w = make_uint2(*reinterpret_cast<const uint32_t*>(src), 0u);
    else
      w = *reinterpret_cast<const uint2*>(src);
    __nv_bfloat16* dst = (is_v ? v_out : k_out) + (t * P.hkv + head) * D + 8 * c;
    *reinterpret_cast<uint4*>(dst) = kv::widen8<BITS>(w, scale, zb);
  }
}

namespace {

Pages view(const sq_kv_pages& p) {
  Pages v{p.k_codes, p.k_scale, p.k_zero, p.v_codes, p.v_scale, p.v_zero, p.num_pages, 0, p.hkv};
  while ((1 << v.lps) < p.page_size) ++v.lps;
  return v;
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
  auto kern = pages.bits == 8 ? append_kernel<8> : append_kernel<4>;
  kern<<<grid_for(T * (P.jq + 2 * P.jk), 8), 256, 0, stream>>>(P);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv_paged_append launch", e);
}

sq_status run_dequant(const sq_kv_pages& pages, const int32_t* table, int width, const int32_t* cu,
                      const int32_t* cached, int B, int64_t T, void* k_out, void* v_out,
                      cudaStream_t stream) {
  auto kern = pages.bits == 8 ? dequant_kernel<8> : dequant_kernel<4>;
  kern<<<grid_for(T * pages.hkv, 8), 256, 0, stream>>>(
      view(pages), Batch{table, cu, cached, width, B, T}, static_cast<__nv_bfloat16*>(k_out),
      static_cast<__nv_bfloat16*>(v_out));
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SQ_OK : host::cuda_fail("kv_paged_dequant launch", e);
}

}  // namespace paged
}  // namespace sq
