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
// Magnitudes are compared as unsigned bit patterns with the sign cleared: the
// order is that of the numbers, infinities and NaN above all finite ones.
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

__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

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
__device__ __forceinline__ uint32_t e4m3_byte(float v) { return e4m3x4(v, 0.0f, 0.0f, 0.0f) & 0xFFu; }

// The value of a finite E4M3 byte.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  const uint32_t e = (b >> 3) & 15u, m = b & 7u;
  const float v = e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0.001953125f;
  return (b & 0x80u) ? -v : v;
}

// Eight floats -> eight E2M1 codes (nearest even, saturated to 6), the first
// in the low four bits.  cvt puts its first source in the upper half.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// How a group's values become codes.
struct GroupScale {
  float scale;     // as stored (fp32 scales), or the number behind `byte`
  uint32_t byte;   // as stored (E8M0, E4M3 scales)
  float inv;       // 1 / unit
  float unit;      // what a code of 1 stands for
  int mode;        // 0: multiply by inv; 1: divide by unit (inv may overflow); 2: not finite
};

// amax_bits: the group's largest magnitude; g: the scale per tensor (E4M3 scales).
template <Codes C, Scales S>
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits, float g) {
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
    r.scale = amax_bits ? fmaxf(__fdiv_rn(amax, qmax<C>()), __uint_as_float(1u)) : 1.0f;
    r.unit = r.scale;
    r.inv = __frcp_rn(r.unit);
    if (r.unit < 1.17549435e-38f) r.mode = 1;   // below 2^-126 the reciprocal may overflow
  } else if (S == Scales::kE8M0) {
    const int k = amax_bits ? ceil_exp(__fdiv_rn(amax, qmax<C>())) : 0;
    r.byte = static_cast<uint32_t>(k + 127);
    r.scale = r.unit = exp2i(k);
    r.inv = exp2i(-k);                          // both exact: no rounding before the code's
  } else {
    r.byte = amax_bits ? e4m3_byte(__fdiv_rn(amax, __fmul_rn(6.0f, g))) : 0x38u;
    if (r.byte == 0) r.byte = 1;                // 2^-9: a group this small still has codes
    r.scale = e4m3_value(r.byte);
    r.unit = __fmul_rn(r.scale, g);
    r.inv = __frcp_rn(r.unit);
    if (!(r.unit > 7.9e-31f && r.unit < 1.2e30f)) r.mode = 1;   // outside 2^+-100
  }
  return r;
}

// Eight values -> codes: two words of bytes (INT8, E4M3) or one word (E2M1).
template <Codes C, Scales S>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], const GroupScale& g) {
  float v[8];
  if (g.mode == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (C == Codes::kInt8) {
        v[i] = y[i];
      } else if (C == Codes::kE2M1 && S == Scales::kE4M3) {
        // the quotient y / unit correctly rounded: one Newton step on the
        // product with the rounded reciprocal.  Values and scales of few bits
        // meet exact ties, which the product alone would miss.  (With the
        // signs this way round a zero keeps its own.)
        const float q = __fmul_rn(y[i], g.inv);
        v[i] = fmaf(-fmaf(q, g.unit, -y[i]), g.inv, q);
      } else {
        v[i] = __fmul_rn(y[i], g.inv);
      }
    }
    if (C == Codes::kInt8) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = quant_bits(v[i], g.inv);
      return make_uint2(pack_low_bytes(b[0], b[1], b[2], b[3]), pack_low_bytes(b[4], b[5], b[6], b[7]));
    }
  } else if (g.mode == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(__fdiv_rn(y[i], g.unit), -qmax<C>()), qmax<C>());
    if (C == Codes::kInt8) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = quant_bits(v[i], 1.0f);
      return make_uint2(pack_low_bytes(b[0], b[1], b[2], b[3]), pack_low_bytes(b[4], b[5], b[6], b[7]));
    }
  } else {
    return make_uint2(0u, 0u);
  }
  if (C == Codes::kE2M1) return make_uint2(e2m1x8(v), 0u);
  return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// Byte offset of the scale of (row, group) in the tiled layout the product
// reads: tiles of 128 rows x 4 groups, `tiles_k` of them side by side.
__device__ __forceinline__ int64_t tiled_scale(int64_t row, int32_t group, int32_t tiles_k) {
  return ((row >> 7) * tiles_k + (group >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (group & 3);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

}  // namespace quant
}  // namespace sdq
