// Vectors of 8 bf16 values, and their quantisation to e4m3 over a shared scale.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace upipe {

struct V8 {
  float v[8];
};

__device__ __forceinline__ V8 unpack8(const uint4& q) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
  V8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f.v[2 * i] = t.x;
    f.v[2 * i + 1] = t.y;
  }
  return f;
}

__device__ __forceinline__ uint4 pack8(const V8& f) {
  return make_uint4(pack_bf16(f.v[0], f.v[1]), pack_bf16(f.v[2], f.v[3]), pack_bf16(f.v[4], f.v[5]),
                    pack_bf16(f.v[6], f.v[7]));
}

// Bits of the largest magnitude of 8 values (as unsigned integers: NaN > infinity > numbers).
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float m;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(const V8& f) {
  const float m = max3_abs(max3_abs(f.v[0], f.v[1], f.v[2]), f.v[3], f.v[4]);
  return __float_as_uint(max3_abs(max3_abs(m, f.v[5], f.v[6]), f.v[7], 0.f));
}
// The same of bf16 pairs, which need not be unpacked for it: the larger magnitudes of two pairs (with any signs),
// and the larger of a pair's as the bits of an fp32.
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
__device__ __forceinline__ uint32_t amax2(const uint4& v) { return amax2(amax2(v.x, v.y), amax2(v.z, v.w)); }
__device__ __forceinline__ uint32_t pair_bits(uint32_t m) { return max((m << 16) & 0x7fffffffu, m & 0x7fff0000u); }

// Scale of a block whose largest magnitude has the given bits: amax / 448 (as a product with the
// rounded 1/448), or 1 for a block below 2^-100, whose e4m3 codes are all zero then.
__device__ __forceinline__ float block_scale(uint32_t bits) {
  const float amax = __uint_as_float(bits);
  return amax < 7.888609052210118e-31f ? 1.f : amax * (1.f / 448.f);
}

// Codes are e4m3(fp32(y / s)), every step exactly rounded: bf16 values over a shared scale meet e4m3's ties often
// (17 m over a largest value of 7 m), and a quotient that is one unit off sends them to either side.  A division
// per value takes 32% more time (norm of 32768 x 4096: 150 -> 199 us), so the quotient Q = y / s is the product
// with 1 / s as the sum hi + lo of two fp32 numbers, fma(y, hi, y * lo): Q (1 + delta) rounded once, |delta| < 2^-43.
// That differs from fp32(Q) only if a midpoint M of two fp32 numbers lies within 2^-43 of Q, and the code only if one
// of the two is a tie t 2^p of e4m3 (t < 32 odd).  M is then m 2^j with m = t 2^k +- 1 < 2^25, k >= 20, and with the
// 24-bit significands Y and S of y and s, |Q - M| / M = |N| / (m S) for the integer N = Y 2^i - m S, i >= 24.  Modulo
// 2^20 N is S or -S, N is not zero (2^24 would divide S), and N < 2^-43 m S < 64.  So only scales whose low 20 bits
// are within 64 of zero, but not zero, are in doubt: one in 8000, and some percent of those of bf16 blocks (largest
// value 7 m).  These, and scales from 2^60 on, are divided by.
struct Divisor {
  float hi, lo;  // lo >= 0, so that a zero keeps its sign
  bool doubt;
};
__device__ __forceinline__ Divisor divisor(float s) {
  const uint32_t bits = __float_as_uint(s), low = bits & 0xfffffu;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  const float hi = __uint_as_float(__float_as_uint(r) - 3u);  // r is off by a unit at most: hi < 1 / s
  const float e = __fmaf_rn(-hi, s, 1.f);
  return Divisor{hi, __fmaf_rn(e, e, e) * hi, !(bits < 0x5d800000u && low - 1u >= 64u && low < 0x100000u - 64u)};
}

// 8 values over the scale, to e4m3 (nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint2 quant8(const V8& f, const Divisor& d) {
  const float2 hi = make_float2(d.hi, d.hi), lo = make_float2(d.lo, d.lo);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = make_float2(f.v[2 * i], f.v[2 * i + 1]);
    w[i] = __nv_cvt_float2_to_fp8x2(__ffma2_rn(y, hi, __fmul2_rn(y, lo)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The same for a scale in doubt, by Markstein's scheme (IBM J. Res. Dev. 34, 1990): with r = fp32(1 / s) and a q
// within a unit of Q (y r after one such step), q + (y - q s) r with both sums fused is fp32(Q).  y and s go to s in
// [1, 2) by a power of two first, so that no difference is subnormal; an infinite scale makes zeros of the numbers, and NaN of the rest.  A
// function of its own: inlined, it cost the callers registers (norm 149 -> 152 us).
static __device__ __noinline__ uint2 quant8_divided(V8 f, float s) {
  float m;
  if (s < 1.3e36f) {  // scales end at 2^128 / 448
    m = __uint_as_float((254u - (__float_as_uint(s) >> 23)) << 23);
    s *= m;
  } else {
    m = s != s ? s : 0.f;
    s = 1.f;
  }
  const float r = -__frcp_rn(s);  // the quotients' negatives, with which zeros come out with the right sign
  const float2 m2 = make_float2(m, m), s2 = make_float2(s, s), r2 = make_float2(r, r);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(make_float2(f.v[2 * i], f.v[2 * i + 1]), m2);
    float2 q = __fmul2_rn(y, r2);
    q = __ffma2_rn(__ffma2_rn(q, s2, y), r2, q);
    q = __ffma2_rn(__ffma2_rn(q, s2, y), r2, q);
    w[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) ^ 0x8080u;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// e4m3 codes as fp32 (exact; NaN stays NaN).
__device__ __forceinline__ float2 e4m3x2(uint16_t q) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(q, __NV_E4M3)));
}
__device__ __forceinline__ V8 e4m3x8(const uint2& q) {
  V8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = e4m3x2((uint16_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1))));
    f.v[2 * i] = t.x;
    f.v[2 * i + 1] = t.y;
  }
  return f;
}

}  // namespace upipe
