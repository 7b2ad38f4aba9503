// Group quantization shared by the kernels that end in codes and scales
// (the RMS norm and the 4-bit quantizer): from a group's largest magnitude to
// its scale, and from values to codes.
//
//   INT8, E4M3 codes   scale = fl32(amax / Qmax) (Qmax 127, 448), or with E8M0
//                      scales the smallest power of two not below it
//   E2M1 codes, E8M0   scale = the smallest power of two not below
//                      fl32(amax / 6); 32 values a group
//   E2M1 codes, E4M3   scale = E4M3(fl32(amax / fl32(6 g))), at least 2^-9; the
//                      group's unit is fl32(scale * g) with g the scale per
//                      tensor; 16 values a group
//   code = round-to-nearest-even of value / unit.  An all-zero group has
//   scale 1.  A group that holds a NaN or an infinity has a NaN scale (fp32
//   NaN, E8M0 0xFF, E4M3 0x7F) and zero codes, so all of it reads back as NaN.
//
// A group's largest magnitude travels as its bits with the sign cleared: their
// unsigned order is that of the numbers, infinities and NaN above all finite
// ones.
//
// These kernels move few bytes a value, so instructions bound them as soon as
// there are about 15 a value: pairs of values go through two-wide fp32
// instructions, quotients are products with a reciprocal and one Newton step.
#pragma once

#include <cstdint>

#include "sdq_ptx.cuh"

namespace sdq {
namespace quant {

enum class Codes { kInt8, kE4M3, kE2M1 };
enum class Scales { kF32, kE8M0, kE4M3 };

constexpr uint32_t kInfBits = 0x7F800000u;

template <Codes C>
__host__ __device__ constexpr float qmax() {
  return C == Codes::kInt8 ? 127.0f : C == Codes::kE4M3 ? 448.0f : 6.0f;
}

// The largest of three magnitudes; a NaN if one of them is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int kPairs>
__device__ __forceinline__ uint32_t amax(const float2 (&y)[kPairs]) {
  float m = amax3(0.0f, y[0].x, y[0].y);
#pragma unroll
  for (int i = 1; i < kPairs; ++i) m = amax3(m, y[i].x, y[i].y);
  return __float_as_uint(m);
}

// The larger magnitudes of two pairs of bf16 numbers, with signs of their own; a
// NaN where one is.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t amax_bf16x2(const uint4& v) {
  return amax_bf16x2(amax_bf16x2(v.x, v.y), amax_bf16x2(v.z, v.w));
}
// One number of a pair without its sign, as the bits of an fp32 number.
__device__ __forceinline__ uint32_t magnitude_lo(uint32_t v) { return (v << 16) & 0x7FFF0000u; }
__device__ __forceinline__ uint32_t magnitude_hi(uint32_t v) { return v & 0x7FFF0000u; }

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}

// 1 / u within an ulp of the rounded reciprocal, for u and 1 / u normal.
__device__ __forceinline__ float reciprocal(float u) {
  const float r = rcp_approx(u);
  return fmaf(fmaf(-u, r, 1.0f), r, r);
}

// a / d correctly rounded, with inv near 1 / d: the remainder of the product is
// exact while it does not underflow.
__device__ __forceinline__ float quotient(float a, float d, float inv) {
  const float q = __fmul_rn(a, inv);
  return fmaf(fmaf(-q, d, a), inv, q);
}

// 2^k for -127 <= k <= 127 (2^-127 is subnormal).
__device__ __forceinline__ float exp2i(int k) {
  return k > -127 ? __int_as_float((k + 127) << 23) : __int_as_float(1 << 22);
}

// The smallest k in [-127, 127] with 2^k >= t, for a finite t > 0.
__device__ __forceinline__ int ceil_exp(float t) {
  const uint32_t b = __float_as_uint(t);
  const int k = static_cast<int>(b >> 23) - 127 + ((b & 0x7FFFFFu) ? 1 : 0);
  if (b <= (1u << 22)) return -127;          // t <= 2^-127
  return k < -126 ? -126 : k > 127 ? 127 : k;   // a subnormal above 2^-127 needs 2^-126
}

// One E4M3 byte (round to nearest even, saturated to 448).
__device__ __forceinline__ uint32_t e4m3_byte(float v) {
  uint32_t r;
  asm("{\n\t.reg .b16 b;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %1, %2;\n\tcvt.u32.u16 %0, b;\n}\n" : "=r"(r) : "f"(0.0f), "f"(v));
  return r;
}

// The value of an E4M3 byte.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  float v;
  asm("{\n\t.reg .b16 b;\n\tcvt.u16.u32 b, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n}\n" : "=r"(h) : "r"(b));
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n}\n" : "=f"(v) : "r"(h));
  return v;
}

// Eight floats -> eight E2M1 codes (nearest even, saturated to 6), the first
// in the low four bits.  cvt puts its first source in the upper half.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

// What the groups of a call share: the divisor of a group's largest magnitude,
// its reciprocal, the scale per tensor, and how far the usual magnitudes reach up
// from kLowBits, as bits.
struct Divisor {
  float d, inv, g;
  uint32_t span;
};
constexpr uint32_t kLowBits = (127u - 60u) << 23, kHighBits = (127u + 60u) << 23;
template <Codes C, Scales S>
__device__ __forceinline__ Divisor divisor(const float* global) {
  Divisor v;
  v.g = S == Scales::kE4M3 && global ? *global : 1.0f;
  v.d = S == Scales::kE4M3 ? __fmul_rn(6.0f, v.g) : qmax<C>();
  v.inv = S == Scales::kE4M3 ? __frcp_rn(v.d) : 1.0f / qmax<C>();
  v.span = S != Scales::kE4M3 || (v.g > 8.7e-19f && v.g < 1.15e18f) ? kHighBits - kLowBits : 0u;
  return v;
}

// How a group's values become codes.
struct GroupScale {
  float scale;     // as stored (fp32 scales), or the number behind `byte`
  uint32_t byte;   // as stored (E8M0, E4M3 scales)
  float inv;       // 1 / unit
  float unit;      // what a code of 1 stands for
  int mode;        // 0: multiply by inv; 1: divide by unit (inv may overflow); 2: not finite
};

// Any group: zero, tiny, huge, not finite.
template <Codes C, Scales S>
__device__ __noinline__ GroupScale group_scale_any(uint32_t amax_bits, Divisor v) {
  GroupScale r;
  r.byte = 0;
  if (amax_bits >= kInfBits) {
    r.scale = __uint_as_float(0x7FC00000u);
    r.byte = S == Scales::kE8M0 ? 0xFFu : 0x7Fu;
    r.inv = 0.0f;
    r.unit = 1.0f;
    r.mode = 2;
    return r;
  }
  const float amax = __uint_as_float(amax_bits);
  r.mode = 0;
  if (S == Scales::kF32) {
    // at least the smallest subnormal, so that a code times the scale stays
    // near the value however small the group is
    r.scale = amax_bits ? fmaxf(__fdiv_rn(amax, v.d), __uint_as_float(1u)) : 1.0f;
    r.unit = r.scale;
    r.inv = __frcp_rn(r.unit);
    if (r.unit < 1.17549435e-38f) r.mode = 1;   // below 2^-126 the reciprocal may overflow
  } else if (S == Scales::kE8M0) {
    const int k = amax_bits ? ceil_exp(__fdiv_rn(amax, v.d)) : 0;
    r.byte = static_cast<uint32_t>(k + 127);
    r.scale = r.unit = exp2i(k);
    r.inv = exp2i(-k);                          // both exact: no rounding before the code's
  } else if (amax_bits == 0) {                  // whatever the scale per tensor: it is 0 where all of the tensor is
    r.byte = 0x38u;
    r.scale = r.unit = r.inv = 1.0f;
  } else {
    r.byte = e4m3_byte(__fdiv_rn(amax, v.d));
    if (r.byte == 0) r.byte = 1;                // 2^-9: a group this small still has codes
    r.scale = e4m3_value(r.byte);
    r.unit = __fmul_rn(r.scale, v.g);
    r.inv = __frcp_rn(r.unit);
    // units outside 2^+-100, or quotients past it: no Newton step on those
    if (!(r.unit > 7.9e-31f && r.unit < 1.2e30f && __fmul_rn(amax, r.inv) < 1.2e30f)) r.mode = 1;
  }
  return r;
}

// Between 2^-60 and 2^60, and with a scale per tensor there too, no step leaves
// the normal range.
__device__ __forceinline__ bool usual(uint32_t amax_bits, const Divisor& v) { return amax_bits - kLowBits < v.span; }

template <Codes C, Scales S>
__device__ __forceinline__ GroupScale group_scale_usual(uint32_t amax_bits, const Divisor& v) {
  GroupScale r;
  r.byte = 0;
  r.mode = 0;
  const float t = quotient(__uint_as_float(amax_bits), v.d, v.inv);
  if (S == Scales::kF32) {
    r.scale = r.unit = t;
    r.inv = reciprocal(t);
  } else if (S == Scales::kE8M0) {
    r.byte = (__float_as_uint(t) + 0x7FFFFFu) >> 23;   // the exponent, one more where the mantissa is not zero
    r.scale = r.unit = __uint_as_float(r.byte << 23);
    r.inv = __uint_as_float((254u - r.byte) << 23);
  } else {
    r.byte = max(e4m3_byte(t), 1u);
    r.scale = e4m3_value(r.byte);
    r.unit = __fmul_rn(r.scale, v.g);
    r.inv = reciprocal(r.unit);
  }
  return r;
}

// amax_bits: the group's largest magnitude.
template <Codes C, Scales S>
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits, const Divisor& v) {
  return usual(amax_bits, v) ? group_scale_usual<C, S>(amax_bits, v) : group_scale_any<C, S>(amax_bits, v);
}

// f with the scale of a group: the usual scales apart, so that what f does with
// them asks no more of what kind they are (4-bit codes along both axes, 8192 x 4096,
// E8M0 scales: 27.1 us with one scale struct for all, 22.4 so).
template <Codes C, Scales S, class F>
__device__ __forceinline__ void with_scale(uint32_t amax_bits, const Divisor& d, F f) {
  if (usual(amax_bits, d))
    f(group_scale_usual<C, S>(amax_bits, d));
  else
    f(group_scale_any<C, S>(amax_bits, d));
}

// v * inv rounded to whole numbers by one fused multiply-add each (quant_bits).
__device__ __forceinline__ uint2 int8x8(const float2 (&v)[4], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __ffma2_rn(v[i], make_float2(inv, inv), make_float2(12582912.0f, 12582912.0f));
    b[2 * i] = __float_as_uint(q.x);
    b[2 * i + 1] = __float_as_uint(q.y);
  }
  return make_uint2(pack_low_bytes(b[0], b[1], b[2], b[3]), pack_low_bytes(b[4], b[5], b[6], b[7]));
}

// Eight values -> codes: two words of bytes (INT8, E4M3) or one word (E2M1).
template <Codes C, Scales S>
__device__ __forceinline__ uint2 codes8(const float2 (&y)[4], const GroupScale& g) {
  if (g.mode == 2) return make_uint2(0u, 0u);
  float2 v[4];
  if (g.mode == 0) {
    if (C == Codes::kInt8) return int8x8(y, g.inv);
    const float2 inv = make_float2(g.inv, g.inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __fmul2_rn(y[i], inv);
      if (C == Codes::kE2M1 && S == Scales::kE4M3) {
        // the quotient y / unit correctly rounded: one Newton step on the
        // product with the reciprocal.  Values and scales of few bits meet exact
        // ties, which the product alone would miss.  (With the signs this way
        // round a zero keeps its own.)
        const float2 rem = __ffma2_rn(v[i], make_float2(g.unit, g.unit), make_float2(-y[i].x, -y[i].y));
        v[i] = __ffma2_rn(make_float2(-rem.x, -rem.y), inv, v[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(fminf(fmaxf(__fdiv_rn(y[i].x, g.unit), -qmax<C>()), qmax<C>()),
                         fminf(fmaxf(__fdiv_rn(y[i].y, g.unit), -qmax<C>()), qmax<C>()));
    if (C == Codes::kInt8) return int8x8(v, 1.0f);
  }
  if (C == Codes::kE2M1) return make_uint2(e2m1x8(v), 0u);
  return make_uint2(e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y), e4m3x4(v[2].x, v[2].y, v[3].x, v[3].y));
}

// Byte offset of the scale of (row, group) in the tiled layout the product
// reads: tiles of 128 rows x 4 groups, `tiles_k` of them side by side.
__device__ __forceinline__ int64_t tiled_scale(int64_t row, int32_t group, int32_t tiles_k) {
  return ((row >> 7) * tiles_k + (group >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (group & 3);
}

}  // namespace quant
}  // namespace sdq
