// What the kernels of norm, rotation and append share: the angle of a position,
// 16-bit values in and out, and packed fp32 arithmetic.
#pragma once
#include <math.h>

#include "attn.cuh"
#include "common.cuh"

namespace exl3 {

// 2^64 * f / (2 pi) modulo 2^64 for 0 <= f < 64.  f = M 2^(e-1086) with M the
// 53-bit mantissa shifted to the top of 64 bits; C = floor(2^66 / (2 pi)), so
// the result is hi64(M C) 2^(e-1024), with a relative error below 2^-62.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f);
  const int e = (int)(u >> 52) & 0x7FF;
  if (e == 0) return 0;
  const uint64_t m = ((u & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) << 11;
  const uint64_t p = __umul64hi(m, 0xA2F9836E4E441529ull);
  const int s = 1024 - e;
  if (s >= 64 || s < -5) return 0;
  const uint64_t t = s >= 0 ? p >> s : p << -s;
  return (u >> 63) ? 0 - t : t;
}

__device__ __forceinline__ float2 cos_sin(int32_t pos, double inv_freq) {
  const uint64_t phase = turns_of(inv_freq) * (uint64_t)(int64_t)pos;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack4(const uint2& r, int bf16, float* v) {
  const uint32_t w[2] = {r.x, r.y};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    if (bf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint2 pack4(const float* v, int bf16) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    if (bf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Two fp32 operations per instruction: this kernel issues ~80 instructions
// per row and lane, and the scalar forms alone would bound it.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

}  // namespace exl3
