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

template <int C>
__device__ __forceinline__ float q8_top() {
  return C == kCodeI8 ? 127.f : 448.f;
}

// Scale from the largest magnitude's bits (a NaN's are above infinity's, which are above every
// finite one's).
template <int C>
__device__ __forceinline__ float q8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
  return __fdiv_rn(fmaxf(__uint_as_float(amax_bits), kQ8Floor), q8_top<C>());
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

// A word of codes of four fp32 values; x becomes what the codes stand for.  The quotient is the
// correctly rounded one: a value beside a rounding border gets the code that any fp32 program
// gives it.
template <int C>
__device__ __forceinline__ uint32_t q8_encode(float (&x)[4], float scale) {
  uint32_t w = 0;
  if (scale != scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = scale;
    return w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fdiv_rn(x[i], scale);
  if constexpr (C == kCodeI8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = __float2int_rn(x[i]);
      w |= static_cast<uint32_t>(c & 0xff) << (8 * i);
      x[i] = static_cast<float>(c) * scale;
    }
  } else {
    w = e4m3_pack(x[0], x[1]) | e4m3_pack(x[2], x[3]) << 16;
    q8_decode<C>(w, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= scale;
  }
  return w;
}

}  // namespace santa
