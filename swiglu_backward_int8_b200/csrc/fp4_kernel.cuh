// Microscaled 4-bit quantization (quant_common.cuh) of bf16 arrays along the
// rows, along the columns (transposed), or both in one pass, and back.
//
// A CTA takes a tile of 128 rows x 128 channels.  Along the rows a thread has 16
// consecutive channels of a row (a group is one lane or two); along the columns
// it has one group of rows of two neighbouring channels, read back from the tile
// in shared memory, and the codes go through shared memory once more so that the
// stores fill 64 bytes of a row.  The scales of a tile are whole 512-byte scale
// tiles (128 rows x 4 groups, or the transposed ones), put together in shared
// memory.
//
// 2 bytes are read and 0.53 or 0.56 written a value and axis.  Along the rows DRAM
// bounds it (8192 x 4096: 14.5 to 15 us in short runs, 86 to 91 % of the measured
// copy's rate); along the columns (E8M0 scales 18.2 us, E4M3 20.1) and both axes
// instructions do (E8M0 scales 21.9 us, 72 %; E4M3 scales, twice the groups and a
// Newton step a quotient, 26 to 27, 60 %): 16 a value, 59 % of the issue slots by 24
// warps, half of them in the half-rate integer pipe, which unpacks, converts and
// compares.  Groups of zeros go the way of unusual scales: a tensor of them takes up
// to a fifth longer (both axes, E8M0 26.5 us, E4M3 29.9).  Reading back: 12.9 us in
// short runs, 15 among other calls.
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

// The scale tiles of a tile, from shared memory: word w of one has the four groups
// of row (w / 4) + 32 (w % 4).  Rows past the last are left alone.
template <int kAtoms>
__device__ __forceinline__ void store_scale_tiles(const uint8_t* sc, uint8_t* out, int64_t first, int64_t last, int rows,
                                                  int t) {
  for (int w = t; w < kAtoms * 128; w += kThreads) {
    const int r = ((w & 127) >> 2) + 32 * (w & 3);
    const int64_t tile = first + (w >> 7);
    if (r < rows && tile < last)
      *reinterpret_cast<uint32_t*>(out + tile * 512 + (w & 127) * 4) = reinterpret_cast<const uint32_t*>(sc)[w];
  }
}

// CTAs a multiprocessor: four, but three where the columns' groups of 32, or both
// axes, need more registers (both axes, E8M0 scales: 22 us with three, 29 with four).
// Rows alone with E8M0 scales spill 48 bytes at four.
template <Scales S, bool kRows, bool kCols>
__global__ void __launch_bounds__(kThreads, kCols && (kRows || S == Scales::kE8M0) ? 3 : 4) quantize_kernel(const QuantParams p) {
  constexpr int G = S == Scales::kE8M0 ? 32 : 16;
  constexpr int kGroups = kTile / G;          // groups of a tile along either axis
  constexpr int kAtoms = kGroups / 4;         // scale tiles of a tile
  constexpr int kPitch = kTile * 2 + 16;      // bytes of a row of the tile
  constexpr int kCodePitch = kTile / 2;       // bytes of a channel's codes: four pieces of 16, swizzled by its number
  __shared__ alignas(16) uint8_t tile[kCols ? kTile * kPitch : 16];
  __shared__ alignas(16) uint8_t ct[kCols ? kTile * kCodePitch : 16];
  __shared__ alignas(16) uint8_t sc[kRows ? kAtoms * 512 : 16], sct[kCols ? kAtoms * 512 : 16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x;
  const int tile_m = blockIdx.x / p.grid_k, tile_k = blockIdx.x - tile_m * p.grid_k;
  const int k0 = tile_k * kTile;
  const int64_t m0 = static_cast<int64_t>(tile_m) * kTile;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(kTile), p.rows - m0));
  const int nch = min(kTile, p.channels - k0);
  const quant::Divisor d = quant::divisor<Codes::kE2M1, S>(p.global);
  const int c16 = (t & 7) * 16;
  constexpr int kStep = kThreads / 8, kPasses = kTile / kStep;   // rows of a pass
  uint4 va[kPasses], vb[kPasses];
  // addresses go on by a pass's rows: a product of 64 bits each costs more than the loads
  const uint8_t* x = p.x + 2 * ((m0 + (t >> 3)) * p.ld_x + k0 + c16);
  uint8_t* q = kRows ? p.q + (m0 + (t >> 3)) * p.ld_q + ((k0 + c16) >> 1) : nullptr;
  const int rows_here = c16 < nch ? nrows - (t >> 3) : 0;   // rows of this thread's pass 0 to the last
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    va[i] = vb[i] = make_uint4(0, 0, 0, 0);
    if (i * kStep < rows_here) {
      va[i] = reinterpret_cast<const uint4*>(x)[0];
      vb[i] = reinterpret_cast<const uint4*>(x)[1];
    }
    x += 2 * kStep * p.ld_x;
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = (t >> 3) + i * kStep;
    if (kCols) {
      // (four lanes of a row begin with their second half: no two hit a bank)
      uint8_t* o = tile + r * kPitch + c16 * 2;
      const bool late = t & 4;
      *reinterpret_cast<uint4*>(o + (late ? 16 : 0)) = late ? vb[i] : va[i];
      *reinterpret_cast<uint4*>(o + (late ? 0 : 16)) = late ? va[i] : vb[i];
    }
    if (kRows) {
      float2 y[4], z[4];
      quant::unpack8(va[i], y);
      quant::unpack8(vb[i], z);
      uint32_t m = quant::amax_bf16x2(quant::amax_bf16x2(va[i]), quant::amax_bf16x2(vb[i]));
      m = max(quant::magnitude_lo(m), quant::magnitude_hi(m));
      if (G == 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      uint32_t byte;
      uint2 codes;
      quant::with_scale<Codes::kE2M1, S>(m, d, [&](const quant::GroupScale& gs) {
        byte = gs.byte;
        codes = make_uint2(quant::codes8<Codes::kE2M1, S>(y, gs).x, quant::codes8<Codes::kE2M1, S>(z, gs).x);
      });
      if (i * kStep < rows_here) *reinterpret_cast<uint2*>(q) = codes;
      q += kStep * p.ld_q;
      const int grp = c16 / G;
      if ((c16 & (G - 1)) == 0)
        sc[(grp >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (grp & 3)] = static_cast<uint8_t>(c16 < nch ? byte : 0u);
    }
  }
  __syncthreads();
  if (kRows)
    store_scale_tiles<kAtoms>(sc, p.s + static_cast<int64_t>(tile_m) * p.tiles_k * 512, tile_k * kAtoms, p.tiles_k, nrows, t);
  if (kCols) {
    const int c = (t & 63) * 2;                 // two channels
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      const int grp = (t >> 6) + 4 * i;         // the group of rows
      uint32_t v[G];
      uint32_t m = 0, n = 0;
#pragma unroll
      for (int e = 0; e < G; ++e) v[e] = *reinterpret_cast<const uint32_t*>(tile + (grp * G + e) * kPitch + c * 2);
#pragma unroll
      for (int e = 0; e < G; e += 2) {
        m = quant::amax_bf16x2(m, v[e]);
        n = quant::amax_bf16x2(n, v[e + 1]);
      }
      m = quant::amax_bf16x2(m, n);
      uint32_t byte[2];
      const bool in = m0 + grp * G < p.rows_padded;      // whole groups: rows_padded is a multiple of 32
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t q[G / 8];
        quant::with_scale<Codes::kE2M1, S>(h ? quant::magnitude_hi(m) : quant::magnitude_lo(m), d, [&](const quant::GroupScale& gs) {
          byte[h] = gs.byte;
#pragma unroll
          for (int w = 0; w < G / 8; ++w) {
            float2 y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = h ? make_float2(bf16_hi(v[w * 8 + 2 * e]), bf16_hi(v[w * 8 + 2 * e + 1]))
                       : make_float2(bf16_lo(v[w * 8 + 2 * e]), bf16_lo(v[w * 8 + 2 * e + 1]));
            q[w] = quant::codes8<Codes::kE2M1, S>(y, gs).x;
          }
        });
        uint8_t* o = ct + (c + h) * kCodePitch;
        if constexpr (G == 32)
          *reinterpret_cast<uint4*>(o + ((grp ^ ((c >> 1) & 3)) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
        else
          *reinterpret_cast<uint2*>(o + (((grp >> 1) ^ ((c >> 1) & 3)) << 4) + (grp & 1) * 8) = make_uint2(q[0], q[1]);
      }
      uint8_t* o = sct + (grp >> 2) * 512 + (grp & 3);
      o[(c & 31) * 16 + (c >> 5) * 4] = static_cast<uint8_t>(in ? byte[0] : 0u);
      o[((c + 1) & 31) * 16 + (c >> 5) * 4] = static_cast<uint8_t>(in ? byte[1] : 0u);
    }
    __syncthreads();
    store_scale_tiles<kAtoms>(sct, p.st + static_cast<int64_t>(tile_k) * p.tiles_m * 512,
                              static_cast<int64_t>(tile_m) * kAtoms, p.tiles_m, nch, t);
#pragma unroll
    for (int i = 0; i < kTile * 4 / kThreads; ++i) {   // 32 rows of a channel: 16 bytes
      const int ch = (t >> 2) + i * (kThreads / 4), part = t & 3;
      if (ch < nch && m0 + part * 32 < p.rows_padded)
        *reinterpret_cast<uint4*>(p.qt + (k0 + ch) * p.ld_qt + (m0 >> 1) + part * 16) =
            *reinterpret_cast<const uint4*>(ct + ch * kCodePitch + ((part ^ ((ch >> 1) & 3)) << 4));
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
  int32_t grid_k;          // strips of 256 channels
};

// Four codes pairs -> eight numbers: two codes of a byte become two fp16 numbers in
// one instruction, exact; times the unit they are rounded once to fp32 and once
// to bf16.
__device__ __forceinline__ uint4 values8(uint32_t w, float unit) {
  uint32_t h[4], o[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n}\n"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h[i]));
    f = __fmul2_rn(f, make_float2(unit, unit));
    o[i] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// What a code of 1 stands for, from a scale's byte.
template <Scales S>
__device__ __forceinline__ float unit_of(uint32_t b, float g) {
  if (S == Scales::kE8M0) return b == 255 ? __uint_as_float(0x7FC00000u) : b == 0 ? quant::exp2i(-127) : __uint_as_float(b << 23);
  return __fmul_rn(quant::e4m3_value(b), g);   // (a NaN byte is a NaN)
}

// A warp takes 256 channels of kDequantRows rows, a lane 8 of them.
constexpr int kDequantRows = 4, kDequantCols = 256;

template <Scales S>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantParams p) {
  constexpr int G = S == Scales::kE8M0 ? 32 : 16;
  grid_dependency_wait();
  grid_launch_dependents();
  const float g = S == Scales::kE4M3 && p.global ? *p.global : 1.0f;
  const int strip = blockIdx.x / p.grid_k;
  const int k = (blockIdx.x - strip * p.grid_k) * kDequantCols + (threadIdx.x & 31) * 8;
  const int64_t row0 = static_cast<int64_t>(strip) * (kThreads / 32 * kDequantRows) + (threadIdx.x >> 5) * kDequantRows;
  if (k >= p.channels) return;
  const uint8_t* q = p.q + row0 * p.ld_q + (k >> 1);
  const uint8_t* s = p.s + quant::tiled_scale(row0, k / G, p.tiles_k);   // a row on: 16 bytes (they share 32 rows)
  uint8_t* out = p.out + 2 * (row0 * p.ld_out + k);
  const int rows = static_cast<int>(min(static_cast<int64_t>(kDequantRows), p.rows - row0));
  uint32_t w[kDequantRows], b[kDequantRows];
#pragma unroll
  for (int i = 0; i < kDequantRows; ++i) {
    if (i < rows) {
      w[i] = *reinterpret_cast<const uint32_t*>(q);
      b[i] = s[16 * i];
    }
    q += p.ld_q;
  }
#pragma unroll
  for (int i = 0; i < kDequantRows; ++i) {
    if (i < rows) *reinterpret_cast<uint4*>(out) = values8(w[i], unit_of<S>(b[i], g));
    out += 2 * p.ld_out;
  }
}

}  // namespace fp4
}  // namespace sdq
