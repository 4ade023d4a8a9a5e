// The asymmetric KV quantizer shared by the contiguous and the paged caches:
// group parameters, exactly rounded codes and their packing, and the exact
// widening of codes back to values.
#pragma once

#include <cuda_bf16.h>

#include "sq_device.cuh"

namespace sq {
namespace kv {

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Asymmetric parameters of a group from its extremes, combined over the
// group's LANES lanes (2 or 4 adjacent lanes in `pmask`):
// scale = (max' - min') / (2^BITS - 1), zero = rint(-min' / scale).
template <int BITS, int LANES = 2>
__device__ __forceinline__ void asym_params(float lo, float hi, unsigned pmask, float& scale,
                                            float& zero) {
  const float top = static_cast<float>((1 << BITS) - 1);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(pmask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(pmask, hi, o));
  }
  lo = fminf(lo, 0.f);
  hi = fmaxf(hi, 0.f);
  scale = __fdiv_rn(hi - lo, top);
  if (scale == 0.f) scale = 1.0f;
  zero = fminf(fmaxf(rintf(__fdiv_rn(-lo, scale)), 0.f), top);
}

// Magic-rounded codes (low mantissa bits hold the code) of 8 elements into
// BITS / 4 words: nibbles at 4 bits, bytes at 8, first element lowest.
template <int BITS>
__device__ __forceinline__ void pack_codes(const uint32_t (&u)[8], uint32_t* out) {
  if (BITS == 4) {
    out[0] = pack8(u);
  } else {
    out[0] = pack4b(u[0], u[1], u[2], u[3]);
    out[1] = pack4b(u[4], u[5], u[6], u[7]);
  }
}

// 8 unsigned codes clamp(rint(x / scale) + zero, 0, 2^BITS - 1), packed; x
// given as 4 float pairs.  The quotient is rounded exactly like IEEE float32
// division: q = x r, e = x - q s, q' = q + e r with r = RN(1 / s), the
// one-step fma correction of Markstein ("IA-64 and Elementary Functions",
// 2000), which yields the correctly rounded quotient when r is the correctly
// rounded reciprocal.  Then rint(q') + zero, clamped to [0, 2^BITS - 1].
// x and s enter scaled by the same power of two u2 (2^64 for a subnormal
// scale, whose reciprocal would overflow, else 1): exact scalings that leave
// the quotient unchanged; s2neg is -s u.
template <int BITS>
__device__ __forceinline__ void ucodes8_div(const f2* x, f2 u2, f2 r2, f2 s2neg, f2 z2,
                                            uint32_t* out) {
  const f2 magic{12582912.f, 12582912.f};       // 1.5 * 2^23: nearest even
  const float lo = 12582912.f, hi = 12582912.f + static_cast<float>((1 << BITS) - 1);
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f2 xs = mul2(x[e], u2);
    const f2 q = mul2(xs, r2);
    const f2 er = fma2(q, s2neg, xs);
    f2 c = add2(add2(fma2(er, r2, q), magic), z2);   // magic + rint(q') + zero, exact
    c.x = fminf(fmaxf(c.x, lo), hi);
    c.y = fminf(fmaxf(c.y, lo), hi);
    u[2 * e] = __float_as_uint(c.x);
    u[2 * e + 1] = __float_as_uint(c.y);
  }
  pack_codes<BITS>(u, out);
}

// bf16((code - zero) * scale) of 8 codes (one word at 4 bits, two at 8).  A
// code becomes a float without a conversion instruction: the bits
// 0x4B000000 | c are 2^23 + c, and subtracting 2^23 + zero leaves c - zero
// exactly; one multiply by the scale then rounds once, as (code - zero) *
// scale does.
template <int BITS>
__device__ __forceinline__ uint4 widen8(uint2 w, float s, float zb) {
  uint32_t t[8];
  if (BITS == 4) {
    const uint32_t lo = w.x & 0x0F0F0F0Fu, hi = (w.x >> 4) & 0x0F0F0F0Fu;
    // element 2j sits in the low nibble of byte j
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[2 * j] = __byte_perm(lo, 0x4B000000u, 0x7440u + j);
      t[2 * j + 1] = __byte_perm(hi, 0x4B000000u, 0x7440u + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[j] = __byte_perm(w.x, 0x4B000000u, 0x7440u + j);
      t[4 + j] = __byte_perm(w.y, 0x4B000000u, 0x7440u + j);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = bf16x2((__uint_as_float(t[2 * e]) - zb) * s, (__uint_as_float(t[2 * e + 1]) - zb) * s);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace kv
}  // namespace sq
