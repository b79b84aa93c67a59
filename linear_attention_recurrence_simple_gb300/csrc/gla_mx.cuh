// MXFP8 arithmetic shared by the quantised pools and tails: E4M3 elements with one E8M0 scale byte
// per block of 32 consecutive values (OCP Microscaling Formats v1.0), the quantisation rule
// described in gla_mxfp8.cu, 16-value pieces (half a block) as the unit of a thread's work.
#pragma once

#include <cuda_fp16.h>

#include "gla_common.cuh"

namespace gla {

// Two E4M3 codes (low byte first in memory) to fp32, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
// Two fp32 values to E4M3 (to nearest, ties to even, saturating), `lo` in the low byte.
__device__ __forceinline__ uint32_t f2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// E8M0 scale byte to its fp32 value 2^(b - 127) (b = 0: the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float e8m0_to_f(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : (b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b << 23));
}
// Shared exponent of a block whose largest magnitude is m (fp32, finite): floor(log2 m) - 8,
// plus one when m's significand exceeds 1.75 (then m 2^-(floor - 8) > 448), clamped to
// [-127, 127]; -127 for zero or subnormal m.
__device__ __forceinline__ int mx_shared_exp(float m) {
  const uint32_t bits = __float_as_uint(m);
  const int E = (int)((bits >> 23) & 0xFFu);
  if (E == 0) return -127;
  const int se = E - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(se, -127);
}
// Pairs of fp32 values through the packed two-lane instructions (each lane rounded as its scalar
// counterpart, so the results are those of the scalar code).
__device__ __forceinline__ uint64_t f2b(float a, float b) { return ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a); }
__device__ __forceinline__ void b2f(uint64_t r, float& a, float& b) {
  a = __uint_as_float((uint32_t)r);
  b = __uint_as_float((uint32_t)(r >> 32));
}
__device__ __forceinline__ uint64_t pmul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pfma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// 2^-se as fp32 (se in [-127, 120]).
__device__ __forceinline__ float pow2_neg(int se) { return __uint_as_float((uint32_t)(127 - se) << 23); }

// 16 fp32 values -> 16 codes (one uint4), given the block's shared exponent.
__device__ __forceinline__ uint4 quantise16(const float (&x)[16], int se) {
  const float inv = pow2_neg(se);
  const uint64_t inv2 = f2b(inv, inv);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y0, y1, y2, y3;
    b2f(pmul(f2b(x[4 * j], x[4 * j + 1]), inv2), y0, y1);
    b2f(pmul(f2b(x[4 * j + 2], x[4 * j + 3]), inv2), y2, y3);
    w[j] = f2_to_e4m3x2(y0, y1) | (f2_to_e4m3x2(y2, y3) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void dequantise16(uint4 c, float scale, float (&x)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = e4m3x2_to_f2(w[j] & 0xFFFFu), b = e4m3x2_to_f2(w[j] >> 16);
    x[4 * j] = a.x * scale;
    x[4 * j + 1] = a.y * scale;
    x[4 * j + 2] = b.x * scale;
    x[4 * j + 3] = b.y * scale;
  }
}
// Largest magnitude of the block whose two 16-value halves sit in lanes t and t ^ 1.
__device__ __forceinline__ float block_max(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
}

template <class T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = reinterpret_cast<const float4*>(p)[j];
    v[4 * j] = f.x;
    v[4 * j + 1] = f.y;
    v[4 * j + 2] = f.z;
    v[4 * j + 3] = f.w;
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[j];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
      v[8 * j + 2 * e] = f.x;
      v[8 * j + 2 * e + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

}  // namespace gla
