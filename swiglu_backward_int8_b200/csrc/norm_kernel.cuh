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
//
// One pass over the arrays, a row in a CTA's registers (several short rows to a
// warp or a CTA); longer rows are read again from L2.  DRAM bounds long calls:
// 16384 x 7168, residual, E4M3 codes, one scale for 128 channels, 127 us in short
// runs, 99 % of the measured copy's rate, and 138 sustained; the backward of 16384 x
// 4096, 87 and 96 us, 94 %, of 16384 x 7168, 168 us in short runs, 86 % (14 warps a
// multiprocessor, by registers).  Rows that are read again: 4096 x 20480 171 us,
// half the rate, the backward 230.  Short calls are bound by the row's latency
// (load, sum over the CTA, scale, store) and the launch: 1 x 7168, 2.9 us; the
// backward of 517 x 7168, 9.2 us.
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
  int64_t rows;
  uint32_t ld_x, ld_residual, ld_h, ld_q, ld_s, ld_y;   // (a row's offset is one 32 x 32 -> 64 bit product)
  int32_t channels, group, groups;   // group 0: the whole row
  int32_t tiles_k;                   // scale tiles along the channels (E2M1)
  int32_t weight_f32;
  float eps, inv_channels;
};

// The offset of a row, in elements.
__device__ __forceinline__ int64_t at(int64_t row, uint32_t ld) {
  return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(row)) * ld);
}

// Sum (or, as bit patterns, largest) over the threads of one row: 4, 8 or 16
// lanes, or whole warps.  red: one word per warp of the CTA.
__device__ __forceinline__ float row_sum(float v, float* red, int row_threads) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < row_threads) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (row_threads <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row_warps = row_threads >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / row_warps * row_warps;
  v = lane < row_warps ? red[first + lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red, int row_threads) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < row_threads) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  if (row_threads <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row_warps = row_threads >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / row_warps * row_warps;
  return __reduce_max_sync(0xffffffffu, lane < row_warps ? red[first + lane] : 0u);
}

// A vector of 16 channels: as loaded, and as 8 pairs of numbers.  (With 8
// channels a vector the addresses, checks and scales took 35 instructions a
// channel, more than the loads' time.)
constexpr int kVec = 16;
struct Vec {
  uint4 a, b;
};
__device__ __forceinline__ Vec load_vec(const uint8_t* p, int32_t k) {
  const uint4* q = reinterpret_cast<const uint4*>(p + 2 * k);
  return {q[0], q[1]};
}
__device__ __forceinline__ void store_vec(uint8_t* p, int32_t k, const Vec& v) {
  uint4* q = reinterpret_cast<uint4*>(p + 2 * k);
  q[0] = v.a;
  q[1] = v.b;
}
using Pairs = float2[8];
__device__ __forceinline__ void unpack(const Vec& v, Pairs& f) {
  const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}
__device__ __forceinline__ Vec pack(const Pairs& f) {
  return {make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                     pack_bf16x2(f[3].x, f[3].y)),
          make_uint4(pack_bf16x2(f[4].x, f[4].y), pack_bf16x2(f[5].x, f[5].y), pack_bf16x2(f[6].x, f[6].y),
                     pack_bf16x2(f[7].x, f[7].y))};
}

// The weights from channel k on.
__device__ __forceinline__ void load_weight(const uint8_t* weight, int f32, int32_t k, Pairs& w) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(weight + 4 * k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = q[i];
      w[2 * i] = make_float2(v.x, v.y);
      w[2 * i + 1] = make_float2(v.z, v.w);
    }
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(weight + 2 * k);
    unpack({q[0], q[1]}, w);
  }
}

// The sum of two bf16 numbers rounded once is what rounding it to fp32 first
// gives: where fp32 would drop bits, the smaller number lies 2^8 below the
// spacing of bf16 and cannot reach a tie.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint4 add_bf16x8(const uint4& a, const uint4& b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

__device__ __forceinline__ float sumsq(const Vec& v) {
  Pairs f;
  float2 s = make_float2(0.0f, 0.0f);
  unpack(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __ffma2_rn(f[i], f[i], s);
  return s.x + s.y;
}

// y of 16 channels, and the largest magnitude among them.
__device__ __forceinline__ uint32_t norm_vec(const Params& p, const Vec& h, int32_t k, float rstd, Pairs& y) {
  Pairs w;
  load_weight(p.weight, p.weight_f32, k, w);
  unpack(h, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul2_rn(__fmul2_rn(y[i], make_float2(rstd, rstd)), w[i]);
  return quant::amax(y);
}

template <Codes C, Scales S>
__device__ __forceinline__ void store_codes(const Params& p, int64_t row, int32_t k, const Pairs& y,
                                            const quant::GroupScale& g) {
  const uint2 a = quant::codes8<C, S>(*reinterpret_cast<const float2(*)[4]>(&y[0]), g);
  const uint2 b = quant::codes8<C, S>(*reinterpret_cast<const float2(*)[4]>(&y[4]), g);
  uint8_t* q = p.q + at(row, p.ld_q);
  if (C == Codes::kE2M1)
    *reinterpret_cast<uint2*>(q + (k >> 1)) = make_uint2(a.x, b.x);
  else
    *reinterpret_cast<uint4*>(q + k) = make_uint4(a.x, a.y, b.x, b.y);
  if (p.y) store_vec(p.y + 2 * at(row, p.ld_y), k, pack(y));
}

template <Codes C, Scales S>
__device__ __forceinline__ void store_scale(const Params& p, int64_t row, int32_t group, const quant::GroupScale& g) {
  if (C == Codes::kE2M1)
    p.s[quant::tiled_scale(row, group, p.tiles_k)] = static_cast<uint8_t>(g.byte);
  else if (S == Scales::kF32)
    reinterpret_cast<float*>(p.s)[at(row, p.ld_s) + group] = g.scale;
  else
    p.s[at(row, p.ld_s) + group] = static_cast<uint8_t>(g.byte);
}

// Threads [0, row_threads) of a CTA take its first row, and so on; short rows
// share a warp.  A thread
// holds a vector of 16 consecutive channels, the next thread the next 16, so a
// group of 16 to 256 channels is 1 to 16 neighbouring lanes of a warp.

// The largest magnitude of a group from that of each lane's vector.
template <Codes C, Scales S>
__device__ __forceinline__ uint32_t group_max(int32_t group, uint32_t m) {
  if (C != Codes::kE2M1 || S == Scales::kE8M0) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // 32 channels at least
  if (C != Codes::kE2M1) {
    if (group > 32) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (group > 64) m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
    if (group > 128) m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
  }
  return m;
}

// The group of channel k, where k begins it; -1 elsewhere.
template <Codes C, Scales S>
__device__ __forceinline__ int32_t group_begun(int32_t group, int32_t k) {
  if (C == Codes::kE2M1) return S == Scales::kE4M3 ? k >> 4 : (k & 31) ? -1 : k >> 5;
  const int shift = 31 - __clz(group);   // a power of two
  return (k & (group - 1)) ? -1 : k >> shift;
}

// 1 / sqrt(mean + eps): the hardware's approximation (2^-22) and one Newton step.
__device__ __forceinline__ float rstd_of(const Params& p, float ss) {
  const float v = fmaf(ss, p.inv_channels, p.eps);
  if (!(v > 1e-36f && v < 1e36f)) return __frsqrt_rn(v);   // zero, tiny, huge, not finite
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return fmaf(fmaf(v * r, -r, 1.0f) * 0.5f, r, r);
}

// Groups that pad the last scale tile: zero, as the product multiplies them
// with zero codes.
template <Codes C>
__device__ __forceinline__ void pad_scales(const Params& p, int64_t row, int t) {
  if (C == Codes::kE2M1 && t < p.tiles_k * 4 - p.groups) p.s[quant::tiled_scale(row, p.groups + t, p.tiles_k)] = 0;
}

// Rows that fit a CTA, a vector a thread.  With kAhead a persistent grid, the
// loads of the next row under way while a row is reduced, normed and stored:
// else a multiprocessor's loads come in bursts with pauses between them.
template <Codes C, Scales S, bool kAhead>
__device__ __forceinline__ void rmsnorm_quant(const Params& p, int row_threads) {
  __shared__ float red[2][2][32];
  grid_dependency_wait();   // inputs may come from the previous kernel in the stream
  grid_launch_dependents();
  const int rows_cta = blockDim.x / row_threads;
  const int t = threadIdx.x % row_threads, k = t * kVec;
  // (a group of a short row has no more lanes than the row)
  const int32_t group = min(p.group, row_threads * kVec);
  const bool in = k < p.channels;
  const quant::Divisor d = quant::divisor<C, S>(p.global);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_cta + threadIdx.x / row_threads;
  Vec x = {}, r = {};
  auto load = [&](int64_t from) {
    if (from >= p.rows || !in) return;
    x = load_vec(p.x + 2 * at(from, p.ld_x), k);
    if (p.residual) r = load_vec(p.residual + 2 * at(from, p.ld_residual), k);
  };
  load(row);
  int flip = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_cta; base < p.rows; base += stride, row += stride) {
    const bool on = in && row < p.rows;
    Vec h = {};
    float ss = 0.0f;
    if (on) {
      h = x;
      if (p.residual) {
        h = {add_bf16x8(x.a, r.a), add_bf16x8(x.b, r.b)};
        store_vec(p.h + 2 * at(row, p.ld_h), k, h);
      }
      ss = sumsq(h);
    }
    if (kAhead) load(row + stride);
    ss = row_sum(ss, red[flip][0], row_threads);
    const float rstd = rstd_of(p, ss);
    if (on && t == 0 && p.rstd) p.rstd[row] = rstd;
    Pairs y = {};
    uint32_t m = on ? norm_vec(p, h, k, rstd, y) : 0;
    const bool whole = C != Codes::kE2M1 && p.group == 0;   // one scale a row
    m = whole ? row_max(m, reinterpret_cast<uint32_t*>(red[flip][1]), row_threads) : group_max<C, S>(group, m);
    flip ^= 1;
    if (on)
      quant::with_scale<C, S>(m, d, [&](const quant::GroupScale& g) {
        const int32_t begun = whole ? (t == 0 ? 0 : -1) : group_begun<C, S>(p.group, k);
        if (begun >= 0) store_scale<C, S>(p, row, begun, g);
        store_codes<C, S>(p, row, k, y, g);
      });
    if (row < p.rows) pad_scales<C>(p, row, t);   // (a short row has fewer vectors than groups to pad)
    if (!kAhead) break;   // one row a thread
  }
}

// Few rows: each has a CTA.
template <Codes C, Scales S>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_quant_kernel(const Params p, int row_threads) {
  rmsnorm_quant<C, S, false>(p, row_threads);
}

// 64 registers: eight warps a quarter of a multiprocessor.  (Two vectors a thread
// and 80 registers, six warps: 160 us for 16384 x 7168 where this took 138.)
constexpr int kAheadRegs = 64;

template <Codes C, Scales S>
__global__ void __maxnreg__(kAheadRegs) rmsnorm_quant_rows_kernel(const Params p, int row_threads) {
  rmsnorm_quant<C, S, true>(p, row_threads);
}

// Longer rows: h is read again (from L2) for the second pass, and with a scale
// a row for a third.
template <Codes C, Scales S>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_quant_long_kernel(const Params p) {
  __shared__ float red[2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x, step = blockDim.x * kVec;
  const int64_t row = blockIdx.x;
  const quant::Divisor d = quant::divisor<C, S>(p.global);
  const uint8_t* hb = p.residual ? p.h + 2 * at(row, p.ld_h) : p.x + 2 * at(row, p.ld_x);
  float ss = 0.0f;
  for (int k = t * kVec; k < p.channels; k += step) {
    Vec h = load_vec(p.x + 2 * at(row, p.ld_x), k);
    if (p.residual) {
      const Vec r = load_vec(p.residual + 2 * at(row, p.ld_residual), k);
      h = {add_bf16x8(h.a, r.a), add_bf16x8(h.b, r.b)};
      store_vec(p.h + 2 * at(row, p.ld_h), k, h);
    }
    ss += sumsq(h);
  }
  ss = row_sum(ss, red[0], blockDim.x);
  const float rstd = rstd_of(p, ss);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
  const bool whole = C != Codes::kE2M1 && p.group == 0;
  quant::GroupScale g;
  if (whole) {
    uint32_t m = 0;
    for (int k = t * kVec; k < p.channels; k += step) {
      Pairs y;
      m = max(m, norm_vec(p, load_vec(hb, k), k, rstd, y));
    }
    g = quant::group_scale<C, S>(row_max(m, reinterpret_cast<uint32_t*>(red[1]), blockDim.x), d);
    if (t == 0) store_scale<C, S>(p, row, 0, g);
  }
  for (int k0 = 0; k0 < p.channels; k0 += step) {   // (all lanes of a warp: they reduce together)
    const int k = k0 + t * kVec;
    const bool on = k < p.channels;
    Pairs y = {};
    const uint32_t m = on ? norm_vec(p, load_vec(hb, k), k, rstd, y) : 0;
    if (!whole) g = quant::group_scale<C, S>(group_max<C, S>(p.group, m), d);
    if (on) {
      const int32_t begun = whole ? -1 : group_begun<C, S>(p.group, k);
      if (begun >= 0) store_scale<C, S>(p, row, begun, g);
      store_codes<C, S>(p, row, k, y, g);
    }
  }
  pad_scales<C>(p, row, t);
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
  int64_t rows;
  uint32_t ld_gy, ld_h, ld_gh, ld_gx;
  int32_t channels, weight_f32, parts;
  float inv_channels;
};

// CTA b takes rows b, b + parts, ... and adds their grad_y n to its own row of
// `part`, in that order; grad_weight_kernel adds the rows of `part` in theirs.
// No atomics: the result does not depend on timing.

__device__ __forceinline__ void load_weight8(const uint8_t* weight, int f32, int32_t k, float2 (&w)[4]) {
  if (f32) {
    const float4 a = *reinterpret_cast<const float4*>(weight + 4 * k);
    const float4 b = *(reinterpret_cast<const float4*>(weight + 4 * k) + 1);
    w[0] = make_float2(a.x, a.y);
    w[1] = make_float2(a.z, a.w);
    w[2] = make_float2(b.x, b.y);
    w[3] = make_float2(b.z, b.w);
  } else {
    quant::unpack8(*reinterpret_cast<const uint4*>(weight + 2 * k), w);
  }
}

// grad_x of eight channels, grad_y n of them added to acc.  mean: the row's mean of
// grad_y w n.  (In the formula's own order: rstd^3, which would save forming n
// first, leaves fp32's range while the result is well inside.)
__device__ __forceinline__ void backward8(const BwdParams& p, uint8_t* gx, int32_t k, const uint4& gyv, const uint4& hv,
                                          const uint4& ghv, float rstd, float mean, float2 (&acc)[4]) {
  float2 gy[4], h[4], gh[4], w[4];
  quant::unpack8(gyv, gy);
  quant::unpack8(hv, h);
  quant::unpack8(ghv, gh);
  load_weight8(p.weight, p.weight_f32, k, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 r = make_float2(rstd, rstd);
    const float2 n = __fmul2_rn(h[i], r);
    const float2 d = __ffma2_rn(n, make_float2(-mean, -mean), __fmul2_rn(gy[i], w[i]));
    gh[i] = __ffma2_rn(d, r, gh[i]);
    acc[i] = __ffma2_rn(gy[i], n, acc[i]);
  }
  *reinterpret_cast<uint4*>(gx + 2 * k) = quant::pack8(gh);
}

__device__ __forceinline__ float dot8(const BwdParams& p, int32_t k, const uint4& gyv, const uint4& hv) {
  float2 gy[4], h[4], w[4], s = make_float2(0.0f, 0.0f);
  quant::unpack8(gyv, gy);
  quant::unpack8(hv, h);
  load_weight8(p.weight, p.weight_f32, k, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __ffma2_rn(__fmul2_rn(gy[i], w[i]), h[i], s);
  return s.x + s.y;
}

// mean(grad_y w n), from the row's sum of grad_y w h.
__device__ __forceinline__ float backward_mean(const BwdParams& p, float rstd, float dot) {
  return rstd * (dot * p.inv_channels);
}

// Rows that fit the registers, kVecs vectors a thread: grad_y and h of the next
// row are loaded ahead, grad_h while the row's sum is added up.  Short rows go
// several to a CTA (threads [0, row_threads) the first, and so on); its sums are
// put together at the end, in the rows' order.
// (kSeveral false: one row, and the compiler knows.)
template <int kVecs, bool kSeveral>
__device__ __forceinline__ void rmsnorm_backward(const BwdParams& p, int threads) {
  __shared__ float red[2][32];
  extern __shared__ float sums[];   // [rows of the CTA][channels], for several rows
  grid_dependency_wait();
  grid_launch_dependents();
  const int row_threads = kSeveral ? threads : blockDim.x;
  const int rows_cta = kSeveral ? blockDim.x / row_threads : 1;
  const int t = kSeveral ? threadIdx.x % row_threads : threadIdx.x, mine = kSeveral ? threadIdx.x / row_threads : 0;
  const int64_t stride = static_cast<int64_t>(p.parts) * rows_cta;
  float2 acc[kVecs][4] = {};
  uint4 gn[kVecs], hn[kVecs];
  auto load = [&](int64_t row) {
    if (row >= p.rows) return;
    const uint8_t* gy = p.gy + 2 * at(row, p.ld_gy);
    const uint8_t* h = p.h + 2 * at(row, p.ld_h);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = (t + i * row_threads) * 8;
      if (k < p.channels) {
        gn[i] = *reinterpret_cast<const uint4*>(gy + 2 * k);
        hn[i] = *reinterpret_cast<const uint4*>(h + 2 * k);
      }
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_cta + mine;
  load(row);
  int flip = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows_cta; base < p.rows; base += stride, row += stride) {
    const bool on = !kSeveral || row < p.rows;
    const float rstd = on ? p.rstd[row] : 0.0f;
    const uint8_t* gh = p.gh ? p.gh + 2 * at(row, p.ld_gh) : nullptr;
    uint8_t* gx = p.gx + 2 * at(row, p.ld_gx);
    uint4 gv[kVecs], hv[kVecs], rv[kVecs];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = (t + i * row_threads) * 8;
      gv[i] = gn[i];
      hv[i] = hn[i];
      rv[i] = make_uint4(0, 0, 0, 0);
      if (on && k < p.channels) {
        if (gh) rv[i] = *reinterpret_cast<const uint4*>(gh + 2 * k);
        dot += dot8(p, k, gv[i], hv[i]);
      }
    }
    load(row + stride);
    dot = row_sum(dot, red[flip], row_threads);
    flip ^= 1;
    const float mean = backward_mean(p, rstd, dot);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = (t + i * row_threads) * 8;
      if (on && k < p.channels) backward8(p, gx, k, gv[i], hv[i], rv[i], rstd, mean, acc[i]);
    }
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.channels;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (t + i * row_threads) * 8;
    if (k < p.channels) {
      float4* q = reinterpret_cast<float4*>((rows_cta > 1 ? sums + mine * p.channels : part) + k);
      q[0] = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
      q[1] = make_float4(acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y);
    }
  }
  if (rows_cta > 1) {
    __syncthreads();
    for (int k = threadIdx.x; k < p.channels; k += blockDim.x) {
      float s = sums[k];
      for (int r = 1; r < rows_cta; ++r) s += sums[r * p.channels + k];
      part[k] = s;
    }
  }
}

// Registers a thread, and with them warps a quarter of a multiprocessor: 8, 6, 4.
// (Two vectors in several rows a CTA spill 8 bytes, four vectors 48: a register
// more a thread is two warps fewer.)
constexpr int backward_regs(int vecs) { return vecs == 1 ? 64 : vecs == 2 ? 80 : 128; }

template <int kVecs, bool kSeveral>
__global__ void __maxnreg__(backward_regs(kVecs)) rmsnorm_backward_kernel(const BwdParams p, int row_threads) {
  rmsnorm_backward<kVecs, kSeveral>(p, row_threads);
}

// Calls of few values: one kernel, in which the first CTAs add up grad_weight
// straight from grad_y and h (64 channels each, read once more, from L2) while
// the others do the rows.  No partial sums, no second launch: 517 x 7168 9.2 us
// instead of 11.3, 256 x 4096 3.9 instead of 6.8.
constexpr int kWeightCols = 64;

// (40 registers for a vector a thread: 512 x 4096 7.6 -> 6.4 us)
template <int kVecs>
__global__ void __maxnreg__(kVecs == 1 ? 40 : 64) rmsnorm_backward_few_kernel(const BwdParams p, int row_threads,
                                                                           int weight_ctas) {
  __shared__ float red[32];
  __shared__ float sums[32][kWeightCols];
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) < weight_ctas) {
    // a thread has 8 channels of every (threads / 8)th row; the four rows of a
    // warp are added, then the warps' sums in their order
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int k = blockIdx.x * kWeightCols + (lane & 7) * 8;
    float2 acc[4] = {};
    if (k < p.channels) {
#pragma unroll(kVecs == 1 ? 2 : 4)
      for (int64_t row = threadIdx.x >> 3; row < p.rows; row += blockDim.x >> 3) {
        float2 gy[4], h[4];
        quant::unpack8(*reinterpret_cast<const uint4*>(p.gy + 2 * (at(row, p.ld_gy) + k)), gy);
        quant::unpack8(*reinterpret_cast<const uint4*>(p.h + 2 * (at(row, p.ld_h) + k)), h);
        const float r = p.rstd[row];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __ffma2_rn(gy[i], __fmul2_rn(h[i], make_float2(r, r)), acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, 8);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, 8);
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, 16);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, 16);
      if (lane < 8) *reinterpret_cast<float2*>(&sums[warp][lane * 8 + 2 * i]) = acc[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < kWeightCols; c += blockDim.x) {
      float s = sums[0][c];
      for (int i = 1; i < warps; ++i) s += sums[i][c];
      if (blockIdx.x * kWeightCols + c < p.channels) p.gw[blockIdx.x * kWeightCols + c] = s;
    }
    return;
  }
  const int t = threadIdx.x % row_threads;
  const int64_t row = static_cast<int64_t>(blockIdx.x - weight_ctas) * (blockDim.x / row_threads) + threadIdx.x / row_threads;
  const bool on = row < p.rows;
  const float rstd = on ? p.rstd[row] : 0.0f;
  uint4 gv[kVecs], hv[kVecs], rv[kVecs];
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (t + i * row_threads) * 8;
    gv[i] = hv[i] = rv[i] = make_uint4(0, 0, 0, 0);
    if (on && k < p.channels) {
      gv[i] = *reinterpret_cast<const uint4*>(p.gy + 2 * (at(row, p.ld_gy) + k));
      hv[i] = *reinterpret_cast<const uint4*>(p.h + 2 * (at(row, p.ld_h) + k));
      if (p.gh) rv[i] = *reinterpret_cast<const uint4*>(p.gh + 2 * (at(row, p.ld_gh) + k));
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (t + i * row_threads) * 8;
    if (on && k < p.channels) dot += dot8(p, k, gv[i], hv[i]);
  }
  dot = row_sum(dot, red, row_threads);
  const float mean = backward_mean(p, rstd, dot);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int k = (t + i * row_threads) * 8;
    float2 unused[4] = {};
    if (on && k < p.channels) backward8(p, p.gx + 2 * at(row, p.ld_gx), k, gv[i], hv[i], rv[i], rstd, mean, unused);
  }
}

// Longer rows: read twice, the sums of grad_y n in memory between rows (a
// thread's own).
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_backward_long_kernel(const BwdParams p) {
  __shared__ float red[2][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x, step = blockDim.x * 8;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.channels;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const float rstd = p.rstd[row];
    const uint8_t *gy = p.gy + 2 * at(row, p.ld_gy), *h = p.h + 2 * at(row, p.ld_h);
    const uint8_t* gh = p.gh ? p.gh + 2 * at(row, p.ld_gh) : nullptr;
    uint8_t* gx = p.gx + 2 * at(row, p.ld_gx);
    float dot = 0.0f;
    for (int k = t * 8; k < p.channels; k += step)
      dot += dot8(p, k, *reinterpret_cast<const uint4*>(gy + 2 * k), *reinterpret_cast<const uint4*>(h + 2 * k));
    dot = row_sum(dot, red[flip], blockDim.x);
    flip ^= 1;
    const float mean = backward_mean(p, rstd, dot);
    for (int k = t * 8; k < p.channels; k += step) {
      float4* q = reinterpret_cast<float4*>(part + k);
      float2 acc[4] = {};
      if (row != blockIdx.x) {
        const float4 u = q[0], v = q[1];
        acc[0] = make_float2(u.x, u.y);
        acc[1] = make_float2(u.z, u.w);
        acc[2] = make_float2(v.x, v.y);
        acc[3] = make_float2(v.z, v.w);
      }
      backward8(p, gx, k, *reinterpret_cast<const uint4*>(gy + 2 * k), *reinterpret_cast<const uint4*>(h + 2 * k),
                gh ? *reinterpret_cast<const uint4*>(gh + 2 * k) : make_uint4(0, 0, 0, 0), rstd, mean, acc);
      q[0] = make_float4(acc[0].x, acc[0].y, acc[1].x, acc[1].y);
      q[1] = make_float4(acc[2].x, acc[2].y, acc[3].x, acc[3].y);
    }
  }
}

// gw[k] = sum over the rows of part: 32 columns a CTA, a warp takes every 32nd
// row, then the 32 sums are added as a tree.
__global__ void __launch_bounds__(1024) grad_weight_kernel(const float* part, float* gw, int32_t parts, int32_t channels) {
  __shared__ float sum[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (k < channels) {
#pragma unroll 4
    for (int r = warp; r < parts; r += 32) s += part[static_cast<int64_t>(r) * channels + k];
  }
  sum[warp][lane] = s;
  __syncthreads();
  s = sum[lane][warp];   // column `warp`, the sum of warp `lane`
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0 && blockIdx.x * 32 + warp < channels) gw[blockIdx.x * 32 + warp] = s;
}

}  // namespace norm
}  // namespace sdq
