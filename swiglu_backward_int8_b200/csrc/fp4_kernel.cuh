// Microscaled 4-bit quantization (quant_common.cuh) of bf16 arrays along the
// rows, along the columns (transposed), or both in one pass, and back.
//
// A CTA takes a tile of 128 rows x 128 channels.  Along the rows a thread has 8
// consecutive channels of a row (a group is 4 or 2 neighbouring lanes); along
// the columns a thread has one group of rows of two neighbouring channels,
// read back from the tile in shared memory.  The scales of a tile are whole
// 512-byte scale tiles (128 rows x 4 groups, or the transposed ones), put
// together in shared memory.
#pragma once

#include <cstdint>

#include "quant_common.cuh"

namespace sdq {
namespace fp4 {

using quant::Codes;
using quant::Scales;

constexpr int kTile = 128;
constexpr int kThreads = 256;

struct QuantParams {
  const uint8_t* x;        // bf16 rows, ld_x elements apart
  uint8_t* q;              // codes along the rows, ld_q bytes apart; or null
  uint8_t* s;              // their scale tiles
  uint8_t* qt;             // codes along the columns, ld_qt bytes apart; or null
  uint8_t* st;
  const float* global;     // the scale per tensor (E4M3 scales) or null
  int64_t rows, ld_x, ld_q, ld_qt;
  int64_t rows_padded;     // rows up to a multiple of 32: the length of qt's rows in codes
  int32_t channels;
  int32_t tiles_k;         // scale tiles along the channels
  int32_t grid_k;          // tiles along the channels
  int64_t tiles_m;         // scale tiles along the rows (of st)
};

template <Scales S, bool kRows, bool kCols>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantParams p) {
  constexpr int G = S == Scales::kE8M0 ? 32 : 16;
  constexpr int kGroups = kTile / G;          // groups of a tile along either axis
  constexpr int kAtoms = kGroups / 4;         // scale tiles of a tile
  constexpr int kPitch = kTile * 2 + 16;      // bytes of a row of the tile
  __shared__ alignas(16) uint8_t tile[kCols ? kTile * kPitch : 16];
  __shared__ alignas(16) uint8_t sc[kRows ? kAtoms * 512 : 16], sct[kCols ? kAtoms * 512 : 16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const int tile_m = blockIdx.x / p.grid_k, tile_k = blockIdx.x - tile_m * p.grid_k;
  const int k0 = tile_k * kTile;
  const int64_t m0 = static_cast<int64_t>(tile_m) * kTile;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(kTile), p.rows - m0));
  const int nch = min(kTile, p.channels - k0);
  const quant::Divisor g = quant::divisor<Codes::kE2M1, S>(p.global);
  const int c8 = (t & 15) * 8;
#pragma unroll
  for (int i = 0; i < kTile * 16 / kThreads; ++i) {
    const int r = (t >> 4) + i * (kThreads / 16);
    uint4 v = make_uint4(0, 0, 0, 0);
    const bool act = r < nrows && c8 < nch;
    if (act) v = *reinterpret_cast<const uint4*>(p.x + 2 * ((m0 + r) * p.ld_x + k0 + c8));
    if (kCols) *reinterpret_cast<uint4*>(tile + r * kPitch + c8 * 2) = v;
    if (kRows) {
      float2 y[4];
      quant::unpack8(v, y);
      uint32_t m = quant::amax(y);
#pragma unroll
      for (int d = 1; d < G / 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      const quant::GroupScale gs = quant::group_scale<Codes::kE2M1, S>(m, g);
      if (act) *reinterpret_cast<uint32_t*>(p.q + (m0 + r) * p.ld_q + ((k0 + c8) >> 1)) = quant::codes8<Codes::kE2M1, S>(y, gs).x;
      const int grp = c8 / G;
      if ((c8 & (G - 1)) == 0)
        sc[(grp >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (grp & 3)] = static_cast<uint8_t>(c8 < nch ? gs.byte : 0u);
    }
  }
  __syncthreads();
  if (kRows) {
    // word w of a scale tile: the four groups of row (w / 4) + 32 (w % 4)
    for (int w = t; w < kAtoms * 128; w += kThreads) {
      const int atom = w >> 7, r = ((w & 127) >> 2) + 32 * (w & 3);
      const int tk = tile_k * kAtoms + atom;
      if (r < nrows && tk < p.tiles_k)
        *reinterpret_cast<uint32_t*>(p.s + (static_cast<int64_t>(tile_m) * p.tiles_k + tk) * 512 + (w & 127) * 4) =
            reinterpret_cast<const uint32_t*>(sc)[w];
    }
  }
  if (kCols) {
    const int c = (t & 63) * 2;                 // two channels
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      const int grp = (t >> 6) + 4 * i;         // the group of rows
      uint32_t v[G];
      float ma = 0.0f, mb = 0.0f;
#pragma unroll
      for (int e = 0; e < G; ++e) v[e] = *reinterpret_cast<const uint32_t*>(tile + (grp * G + e) * kPitch + c * 2);
#pragma unroll
      for (int e = 0; e < G; e += 2) {
        ma = quant::amax3(ma, bf16_lo(v[e]), bf16_lo(v[e + 1]));
        mb = quant::amax3(mb, bf16_hi(v[e]), bf16_hi(v[e + 1]));
      }
      const quant::GroupScale ga = quant::group_scale<Codes::kE2M1, S>(__float_as_uint(ma), g);
      const quant::GroupScale gb = quant::group_scale<Codes::kE2M1, S>(__float_as_uint(mb), g);
      const int64_t row = m0 + grp * G;
      const bool in = row < p.rows_padded;      // whole groups: rows_padded is a multiple of 32
      uint32_t qa[G / 8], qb[G / 8];
#pragma unroll
      for (int w = 0; w < G / 8; ++w) {
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = make_float2(bf16_lo(v[w * 8 + 2 * e]), bf16_lo(v[w * 8 + 2 * e + 1]));
        qa[w] = quant::codes8<Codes::kE2M1, S>(y, ga).x;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = make_float2(bf16_hi(v[w * 8 + 2 * e]), bf16_hi(v[w * 8 + 2 * e + 1]));
        qb[w] = quant::codes8<Codes::kE2M1, S>(y, gb).x;
      }
      if (in && c < nch) {
        uint8_t* d = p.qt + (k0 + c) * p.ld_qt + (row >> 1);
        if (G == 32) {
          *reinterpret_cast<uint4*>(d) = make_uint4(qa[0], qa[1], qa[G / 8 - 2], qa[G / 8 - 1]);
          *reinterpret_cast<uint4*>(d + p.ld_qt) = make_uint4(qb[0], qb[1], qb[G / 8 - 2], qb[G / 8 - 1]);
        } else {
          *reinterpret_cast<uint2*>(d) = make_uint2(qa[0], qa[1]);
          *reinterpret_cast<uint2*>(d + p.ld_qt) = make_uint2(qb[0], qb[1]);
        }
      }
      uint8_t* o = sct + (grp >> 2) * 512 + (grp & 3);
      o[(c & 31) * 16 + (c >> 5) * 4] = static_cast<uint8_t>(in ? ga.byte : 0u);
      o[((c + 1) & 31) * 16 + (c >> 5) * 4] = static_cast<uint8_t>(in ? gb.byte : 0u);
    }
    __syncthreads();
    for (int w = t; w < kAtoms * 128; w += kThreads) {
      const int atom = w >> 7, r = ((w & 127) >> 2) + 32 * (w & 3);
      const int64_t tm = static_cast<int64_t>(tile_m) * kAtoms + atom;
      if (r < nch && tm < p.tiles_m)
        *reinterpret_cast<uint32_t*>(p.st + (static_cast<int64_t>(tile_k) * p.tiles_m + tm) * 512 + (w & 127) * 4) =
            reinterpret_cast<const uint32_t*>(sct)[w];
    }
  }
}

// ---- back to bf16 -------------------------------------------------------------

struct DequantParams {
  const uint8_t* q;
  const uint8_t* s;
  const float* global;
  uint8_t* out;            // bf16 rows, ld_out elements apart
  int64_t rows, ld_q, ld_out;
  int32_t channels, tiles_k;
};

// The value behind a code: a table lookup in registers (twice the magnitude
// is a nibble of 0x C864 3210), exact; times the unit it is rounded once to
// fp32 and once to bf16.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const float v = static_cast<float>((0xC8643210u >> ((c & 7u) * 4)) & 15u) * 0.5f;
  return (c & 8u) ? -v : v;
}

__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7FC00000u) : quant::exp2i(static_cast<int>(b) - 127);
}

template <Scales S>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantParams p) {
  constexpr int G = S == Scales::kE8M0 ? 32 : 16;
  grid_dependency_wait();
  grid_launch_dependents();
  const float g = S == Scales::kE4M3 && p.global ? *p.global : 1.0f;
  const int64_t vecs = p.channels >> 3;
  const int64_t total = p.rows * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = i / vecs;
    const int32_t k = static_cast<int32_t>(i - row * vecs) * 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p.q + row * p.ld_q + (k >> 1));
    const uint32_t b = p.s[quant::tiled_scale(row, k / G, p.tiles_k)];
    float unit;
    if (S == Scales::kE8M0)
      unit = e8m0_value(b);
    else
      unit = (b & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : __fmul_rn(quant::e4m3_value(b), g);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = pack_bf16x2(e2m1_value(w >> (8 * e)) * unit, e2m1_value(w >> (8 * e + 4)) * unit);
    *reinterpret_cast<uint4*>(p.out + 2 * (row * p.ld_out + k)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace fp4
}  // namespace sdq
