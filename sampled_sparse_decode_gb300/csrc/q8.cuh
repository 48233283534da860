// q8.cuh — rows held in 8 bits: a row of d elements x is d codes c and one fp32 scale s, and stands
// for c s.  s = max(max |x|, 2^-90) / top and c = x / s rounded to the nearest code, ties to even;
// top is 127 for int8 and 448 for e4m3.  The bound below 2^-90 keeps s a normal number (a row of
// zeros gets codes 0); a row that holds an infinity or a NaN gets s = NaN and codes 0, so that all of
// it reads back as NaN.  A scale per (token, head) lets a token be appended without touching the
// rows before it, and multiplies a whole score or weight rather than every element.
#pragma once

#include "common.cuh"

namespace santa {

enum CodeType { kCodeNone = 0, kCodeI8 = 1, kCodeE4M3 = 2 };   // kCodeNone: the activations' type

constexpr float kQ8Floor = 0x1p-90f;

// Largest magnitude; a NaN stays one.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {   // of any sign
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two fp32 values in a register pair, and one instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }
__device__ __forceinline__ float2 halves(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The correctly rounded x / y, `inv` being 1 / y rounded: a product and its correction by the exact
// remainder (P. W. Markstein, IBM J. Res. Dev. 34, 1990).
__device__ __forceinline__ float quotient(float x, float y, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, y, x), inv, q);
}

// A row's scale from its largest magnitude, and the scale's reciprocal: the unit's approximation and one
// Newton step.
struct Scale {
  float s, inv;
};
template <int C>
__device__ __forceinline__ Scale q8_scale(float amax) {
  constexpr float top = C == kCodeI8 ? 127.f : 448.f;
  Scale r;
  r.s = quotient(fmaxf(amax, kQ8Floor), top, 1.f / top);
  if (!(amax <= 3.402823466e38f)) r.s = __uint_as_float(0x7fffffffu);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(r.s));
  r.inv = fmaf(fmaf(-r.s, y, 1.f), y, y);
  return r;
}

// Two e4m3 codes (low byte first) of two fp32 values, and the other way round.
__device__ __forceinline__ uint32_t e4m3_pack(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint16_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
  return make_float2(lo, hi);
}

// The four values of a word of codes.
template <int C>
__device__ __forceinline__ void q8_decode(uint32_t w, float (&x)[4]) {
  if constexpr (C == kCodeI8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
    const float2 a = f16x2_to_f32(e4m3_to_f16x2(static_cast<uint16_t>(w)));
    const float2 b = f16x2_to_f32(e4m3_to_f16x2(static_cast<uint16_t>(w >> 16)));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
}

// A word of codes of four fp32 values of a row with this scale; x becomes the codes' values.  The
// quotients are the correctly rounded ones (see `quotient`), so that a value beside a rounding border gets the
// code that any fp32 program gives it.  int8: adding 1.5 * 2^23 rounds to an integer, ties to even, in the
// low byte.
template <int C>
__device__ __forceinline__ uint32_t q8_encode(uint64_t (&x)[2], const Scale& scale) {
  const uint64_t inv = twice(scale.inv), minus = twice(-scale.s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t q = mul_pair(x[i], inv);
    x[i] = fma_pair(fma_pair(q, minus, x[i]), inv, q);
  }
  uint32_t w;
  if constexpr (C == kCodeI8) {
    constexpr float kMagic = 12582912.f;
    const uint64_t lo = add_pair(x[0], twice(kMagic)), hi = add_pair(x[1], twice(kMagic));
    x[0] = add_pair(lo, twice(-kMagic));
    x[1] = add_pair(hi, twice(-kMagic));
    const float2 a = halves(lo), b = halves(hi);
    w = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                    __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  } else {
    const float2 a = halves(x[0]), b = halves(x[1]);
    w = e4m3_pack(a.x, a.y) | e4m3_pack(b.x, b.y) << 16;
    float v[4];
    q8_decode<C>(w, v);
    x[0] = pair(v[0], v[1]);
    x[1] = pair(v[2], v[3]);
  }
  return scale.s == scale.s ? w : 0u;
}

}  // namespace santa
