// RMS norm with the residual's addition and quantized rows, and its backward.
//
//   h[m, k]  = bf16(x[m, k] + residual[m, k])          (h = x without residual)
//   rstd[m]  = 1 / sqrt(mean_k h^2 + eps)
//   y[m, k]  = h[m, k] * rstd[m] * weight[k]            fp32, not rounded
//   codes and scales of y in groups of channels (quant_common.cuh)
//
//   n        = h * rstd
//   grad_x   = bf16(rstd * (grad_y w - n * mean_k(grad_y w n)) + grad_h)
//   grad_w   = sum_m grad_y n
//
// h is rounded to bf16 before the norm because the backward, and the next
// residual addition, read it so.  Sums, rstd and y stay in fp32.
#pragma once

#include <cstdint>

#include "quant_common.cuh"

namespace sdq {
namespace norm {

using quant::Codes;
using quant::Scales;

constexpr int kMaxThreads = 1024;

struct Params {
  const uint8_t* x;          // bf16 rows, ld_x elements apart
  const uint8_t* residual;   // bf16 or null
  const uint8_t* weight;     // bf16 or fp32 [channels]
  uint8_t* h;                // bf16, written when residual is set
  uint8_t* q;                // codes
  uint8_t* s;                // scales
  uint8_t* y;                // bf16 or null
  float* rstd;               // [rows] or null
  const float* global;       // the scale per tensor (E4M3 scales) or null
  int64_t rows, ld_x, ld_residual, ld_h, ld_q, ld_s, ld_y;
  int32_t channels, group, groups;   // group 0: the whole row
  int32_t tiles_k;                   // scale tiles along the channels (E2M1)
  int32_t weight_f32;
  float eps;
};

// Sum (or, as bit patterns, largest) over the threads of one row.
// red: one word per warp of the CTA.
__device__ __forceinline__ float row_sum(float v, float* red, int row_warps) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (row_warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / row_warps * row_warps;
  v = lane < row_warps ? red[first + lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, int row_warps) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (row_warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / row_warps * row_warps;
  return __reduce_max_sync(0xffffffffu, lane < row_warps ? red[first + lane] : 0u);
}

__device__ __forceinline__ void load_weight8(const Params& p, int32_t k, float (&w)[8]) {
  if (p.weight_f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.weight + 4 * static_cast<int64_t>(k)));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.weight + 4 * static_cast<int64_t>(k)) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
    quant::unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight + 2 * static_cast<int64_t>(k))), w);
  }
}

__device__ __forceinline__ uint4 load_h8(const Params& p, int64_t row, int32_t k) {
  uint4 a = *reinterpret_cast<const uint4*>(p.x + 2 * (row * p.ld_x + k));
  if (p.residual) {
    const uint4 b = *reinterpret_cast<const uint4*>(p.residual + 2 * (row * p.ld_residual + k));
    float f[8], r[8];
    quant::unpack8(a, f);
    quant::unpack8(b, r);
    a = make_uint4(pack_bf16x2(f[0] + r[0], f[1] + r[1]), pack_bf16x2(f[2] + r[2], f[3] + r[3]),
                   pack_bf16x2(f[4] + r[4], f[5] + r[5]), pack_bf16x2(f[6] + r[6], f[7] + r[7]));
    *reinterpret_cast<uint4*>(p.h + 2 * (row * p.ld_h + k)) = a;
  }
  return a;
}

__device__ __forceinline__ float sumsq8(const uint4& a) {
  float f[8], s = 0.0f;
  quant::unpack8(a, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
  return s;
}

__device__ __forceinline__ uint32_t norm8(const Params& p, const uint4& a, int32_t k, float rstd, float (&y)[8]) {
  float w[8];
  load_weight8(p, k, w);
  quant::unpack8(a, y);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = __fmul_rn(__fmul_rn(y[i], rstd), w[i]);
    m = max(m, quant::mag(y[i]));
  }
  return m;
}

template <Codes C, Scales S>
__device__ __forceinline__ void store8(const Params& p, int64_t row, int32_t k, const float (&y)[8],
                                       const quant::GroupScale& g) {
  const uint2 c = quant::codes8<C, S>(y, g);
  if (C == Codes::kE2M1)
    *reinterpret_cast<uint32_t*>(p.q + row * p.ld_q + (k >> 1)) = c.x;
  else
    *reinterpret_cast<uint2*>(p.q + row * p.ld_q + k) = c;
  if (p.y)
    *reinterpret_cast<uint4*>(p.y + 2 * (row * p.ld_y + k)) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

template <Codes C, Scales S>
__device__ __forceinline__ void store_scale(const Params& p, int64_t row, int32_t group, const quant::GroupScale& g) {
  if (C == Codes::kE2M1)
    p.s[quant::tiled_scale(row, group, p.tiles_k)] = static_cast<uint8_t>(g.byte);
  else if (S == Scales::kF32)
    reinterpret_cast<float*>(p.s)[row * p.ld_s + group] = g.scale;
  else
    p.s[row * p.ld_s + group] = static_cast<uint8_t>(g.byte);
}

// Threads [0, row_threads) of a CTA take its first row, and so on.  A thread
// holds vectors of 8 consecutive channels, the next thread the next 8, so a
// group of 16 to 256 channels is 2 to 32 neighbouring lanes of a warp.
// kVecs > 0: the row is in registers, kVecs vectors a thread.  kVecs = 0: any
// length, h read again (from L2) for the second pass and, with a scale per
// row, for a third.
template <Codes C, Scales S, int kVecs>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_quant_kernel(const Params p, int row_threads) {
  __shared__ float red[2][32];
  grid_dependency_wait();   // inputs may come from the previous kernel in the stream
  grid_launch_dependents();
  const int row_warps = row_threads >> 5;
  const int t = threadIdx.x % row_threads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / row_threads) + threadIdx.x / row_threads;
  const bool on = row < p.rows;
  const float g = S == Scales::kE4M3 && p.global ? *p.global : 1.0f;
  uint4 hv[kVecs > 0 ? kVecs : 1];
  float ss = 0.0f;
  if (kVecs > 0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = (t + i * row_threads) * 8;
      hv[i] = make_uint4(0, 0, 0, 0);
      if (on && k < p.channels) {
        hv[i] = load_h8(p, row, k);
        ss += sumsq8(hv[i]);
      }
    }
  } else {
    for (int k = t * 8; on && k < p.channels; k += row_threads * 8) ss += sumsq8(load_h8(p, row, k));
  }
  ss = row_sum(ss, red[0], row_warps);
  const float rstd = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.channels)) + p.eps);
  if (on && t == 0 && p.rstd) p.rstd[row] = rstd;

  const uint8_t* hb = p.residual ? p.h : p.x;
  const int64_t ldh = p.residual ? p.ld_h : p.ld_x;
  const int lanes = p.group >> 3;   // lanes of a group
  const int steps = kVecs > 0 ? kVecs : (p.channels + row_threads * 8 - 1) / (row_threads * 8);
  quant::GroupScale rg;
  if (p.group == 0) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (kVecs > 0 ? kVecs : steps); ++i) {
      const int k = (t + i * row_threads) * 8;
      if (on && k < p.channels) {
        float y[8];
        m = max(m, norm8(p, kVecs > 0 ? hv[kVecs > 0 ? i : 0] : *reinterpret_cast<const uint4*>(hb + 2 * (row * ldh + k)),
                         k, rstd, y));
      }
    }
    rg = quant::group_scale<C, S>(row_max(m, reinterpret_cast<uint32_t*>(red[1]), row_warps), g);
    if (on && t == 0) store_scale<C, S>(p, row, 0, rg);
  }
#pragma unroll
  for (int i = 0; i < (kVecs > 0 ? kVecs : steps); ++i) {
    const int k = (t + i * row_threads) * 8;
    const bool act = on && k < p.channels;
    float y[8] = {};
    uint32_t m = 0;
    if (act)
      m = norm8(p, kVecs > 0 ? hv[kVecs > 0 ? i : 0] : *reinterpret_cast<const uint4*>(hb + 2 * (row * ldh + k)), k,
                rstd, y);
    if (p.group != 0) {
      for (int d = 1; d < lanes; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
      rg = quant::group_scale<C, S>(m, g);
      if (act && (t & (lanes - 1)) == 0) store_scale<C, S>(p, row, k / p.group, rg);
    }
    if (act) store8<C, S>(p, row, k, y, rg);
  }
  // groups that pad the last scale tile: zero, as the product multiplies them with zero codes
  if (C == Codes::kE2M1 && on && t < p.tiles_k * 4 - p.groups)
    p.s[quant::tiled_scale(row, p.groups + t, p.tiles_k)] = 0;
}

// ---- backward ---------------------------------------------------------------

struct BwdParams {
  const uint8_t* gy;       // bf16 rows
  const uint8_t* h;
  const uint8_t* weight;   // bf16 or fp32 [channels]
  const float* rstd;       // [rows]
  const uint8_t* gh;       // bf16 rows or null: the gradient that reaches h from elsewhere
  uint8_t* gx;             // bf16 rows
  float* gw;               // [channels]
  float* part;             // [parts, channels] partial sums of gw
  int64_t rows, ld_gy, ld_h, ld_gh, ld_gx;
  int32_t channels, weight_f32, parts;
};

__device__ __forceinline__ void bwd_weight8(const BwdParams& p, int32_t k, float (&w)[8]) {
  Params q;
  q.weight = p.weight;
  q.weight_f32 = p.weight_f32;
  load_weight8(q, k, w);
}

// CTA b takes rows b, b + parts, ... and adds their grad_y n to its own row of
// `part`, in that order; grad_weight_kernel adds the rows of `part` in theirs.
// No atomics: the result does not depend on timing.
template <int kVecs>
__global__ void __launch_bounds__(kVecs < 2 ? kMaxThreads : 512) rmsnorm_backward_kernel(const BwdParams p) {
  __shared__ float red[2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  float acc[kVecs > 0 ? kVecs : 1][8] = {};
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.channels;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const float rstd = p.rstd[row];
    uint4 gv[kVecs > 0 ? kVecs : 1], hv[kVecs > 0 ? kVecs : 1];
    float dot = 0.0f;
    const int steps = kVecs > 0 ? kVecs : (p.channels + threads * 8 - 1) / (threads * 8);
#pragma unroll
    for (int i = 0; i < (kVecs > 0 ? kVecs : steps); ++i) {
      const int k = (t + i * threads) * 8;
      if (k < p.channels) {
        const uint4 a = *reinterpret_cast<const uint4*>(p.gy + 2 * (row * p.ld_gy + k));
        const uint4 b = *reinterpret_cast<const uint4*>(p.h + 2 * (row * p.ld_h + k));
        float gy[8], h[8], w[8];
        quant::unpack8(a, gy);
        quant::unpack8(b, h);
        bwd_weight8(p, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(gy[e] * w[e], h[e] * rstd, dot);
        if (kVecs > 0) {
          gv[kVecs > 0 ? i : 0] = a;
          hv[kVecs > 0 ? i : 0] = b;
        }
      }
    }
    dot = row_sum(dot, red[flip], warps);
    flip ^= 1;
    const float c = __fdiv_rn(dot, static_cast<float>(p.channels));
#pragma unroll
    for (int i = 0; i < (kVecs > 0 ? kVecs : steps); ++i) {
      const int k = (t + i * threads) * 8;
      if (k < p.channels) {
        const uint4 a = kVecs > 0 ? gv[kVecs > 0 ? i : 0] : *reinterpret_cast<const uint4*>(p.gy + 2 * (row * p.ld_gy + k));
        const uint4 b = kVecs > 0 ? hv[kVecs > 0 ? i : 0] : *reinterpret_cast<const uint4*>(p.h + 2 * (row * p.ld_h + k));
        float gy[8], h[8], w[8], o[8], r[8] = {};
        quant::unpack8(a, gy);
        quant::unpack8(b, h);
        bwd_weight8(p, k, w);
        if (p.gh) quant::unpack8(*reinterpret_cast<const uint4*>(p.gh + 2 * (row * p.ld_gh + k)), r);
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = h[e] * rstd;
          o[e] = fmaf(rstd, fmaf(-n, c, gy[e] * w[e]), r[e]);
          d[e] = gy[e] * n;
        }
        *reinterpret_cast<uint4*>(p.gx + 2 * (row * p.ld_gx + k)) =
            make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
        if (kVecs > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[kVecs > 0 ? i : 0][e] += d[e];
        } else {   // the thread's own 8 sums, in memory
          float4* q = reinterpret_cast<float4*>(part + k);
          float4 u = make_float4(0, 0, 0, 0), v = u;
          if (row != blockIdx.x) { u = q[0]; v = q[1]; }
          q[0] = make_float4(u.x + d[0], u.y + d[1], u.z + d[2], u.w + d[3]);
          q[1] = make_float4(v.x + d[4], v.y + d[5], v.z + d[6], v.w + d[7]);
        }
      }
    }
  }
  if (kVecs > 0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = (t + i * threads) * 8;
      if (k < p.channels) {
        float4* q = reinterpret_cast<float4*>(part + k);
        q[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        q[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
  }
}

// gw[k] = sum over the rows of part: 32 columns a CTA, a warp takes every
// eighth row, then the eight sums are added in order.
__global__ void __launch_bounds__(256) grad_weight_kernel(const float* part, float* gw, int32_t parts, int32_t channels) {
  __shared__ float sum[8][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (k < channels)
    for (int r = warp; r < parts; r += 8) s += part[static_cast<int64_t>(r) * channels + k];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && k < channels) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sum[i][lane];
    gw[k] = s;
  }
}

}  // namespace norm
}  // namespace sdq
