// C ABI of the microscaled 4-bit quantizer and product (declared in
// include/sdq.h): argument validation and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "fp4_kernel.cuh"
#include "fp4_matmul.cuh"
#include "fp4_matmul_pair.cuh"
#include "sdq.h"
#include "sdq_internal.h"

namespace {

using sdq::quant::Scales;

bool misaligned(const void* p, uintptr_t mask) { return reinterpret_cast<uintptr_t>(p) & mask; }

// Exactly one scale format.
bool format_ok(uint32_t f, uint32_t more = 0) {
  if (f & ~(SDQ_FMT_E8M0 | SDQ_FMT_SCALE_E4M3 | more)) return false;
  return ((f & SDQ_FMT_E8M0) != 0) != ((f & SDQ_FMT_SCALE_E4M3) != 0);
}

bool length_ok(int64_t k) { return k >= 1 && k <= SDQ_MAX_K && k % SDQ_FP4_K_MULTIPLE == 0; }
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int group_of(uint32_t f) { return f & SDQ_FMT_E8M0 ? 32 : 16; }
int64_t tiles_of(int64_t k, uint32_t f) { return (k / group_of(f) + 3) / 4; }   // scale tiles along k

int launch(const void* kernel, unsigned grid, unsigned block, size_t smem, cudaStream_t stream, void** args,
           unsigned cluster = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  return e == cudaSuccess ? SDQ_OK : sdq_internal::cuda_fail(e);
}

// Sets a kernel's shared-memory limit once a device.
struct SmemLimit {
  std::once_flag once[64];
  cudaError_t err[64] = {};
  int set(const void* kernel, int bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return sdq_internal::cuda_fail(e);
    if (dev < 0 || dev >= 64) return sdq_internal::cuda_fail(cudaErrorInvalidDevice);
    std::call_once(once[dev], [&] {
      err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    return err[dev] == cudaSuccess ? SDQ_OK : sdq_internal::cuda_fail(err[dev]);
  }
};

template <Scales S>
const void* quantize_kernel(bool rows, bool cols) {
  if (rows && cols) return reinterpret_cast<const void*>(sdq::fp4::quantize_kernel<S, true, true>);
  return rows ? reinterpret_cast<const void*>(sdq::fp4::quantize_kernel<S, true, false>)
              : reinterpret_cast<const void*>(sdq::fp4::quantize_kernel<S, false, true>);
}

// One call of the product, checked.
struct Product {
  const void* a; int64_t ld_a; const void* a_s; const float* a_global;
  const void* b; int64_t ld_b; const void* b_s; const float* b_global;
  void* out; int64_t ld_out;
  int64_t m, n, k;
  uint32_t format;
  cudaStream_t stream;
  int32_t stall_step = -1, stall_rank = -1;   // a test's: sdq_matmul_fp4_test_stall
  uint64_t wait_limit = sdq_internal::wait_limit();
};

// Many tiles: pairs of multiprocessors.
template <Scales S, bool kF32>
int launch_pair(const Product& c, int sms) {
  using Z = sdq::mm4::PairShape<S>;
  const int64_t tiles_k = tiles_of(c.k, c.format);
  sdq::mm4::PairParams p = {};
  p.ga = c.a_global;
  p.gb = c.b_global;
  p.out = static_cast<uint8_t*>(c.out);
  p.ld_out = c.ld_out;
  p.rows_a = c.m;
  p.rows_b = c.n;
  p.codes = static_cast<int32_t>(c.k);
  p.tiles_a = static_cast<int32_t>((c.m + 255) / 256);
  p.tiles_b = static_cast<int32_t>((c.n + sdq::mm4::kN - 1) / sdq::mm4::kN);
  const uintptr_t at = reinterpret_cast<uintptr_t>(c.out) | static_cast<uintptr_t>(c.ld_out * (kF32 ? 4 : 2));
  p.vec = at & 15 ? 0 : 1;
  p.stall_step = c.stall_step;
  p.stall_rank = c.stall_rank;
  p.wait_limit_ns = c.wait_limit;
  if (const int e = sdq_internal::device_status_word(&p.status)) return e;
  CUtensorMap ma, mb, msa, msb, mo = {};
  if (const int e = sdq_internal::make_code_map(&ma, c.a, c.k / 2, c.m, c.ld_a, 128)) return e;
  if (const int e = sdq_internal::make_code_map(&mb, c.b, c.k / 2, c.n, c.ld_b, sdq::mm4::kN / 2)) return e;
  if (const int e = sdq_internal::make_scale_map(&msa, c.a_s, tiles_k, (c.m + 127) / 128, Z::kScaleTiles)) return e;
  if (const int e = sdq_internal::make_scale_map(&msb, c.b_s, tiles_k, (c.n + 127) / 128, Z::kScaleTiles)) return e;
  if (p.vec)
    if (const int e = sdq_internal::make_out_map(&mo, c.out, kF32, c.n, c.m, c.ld_out)) return e;
  const void* fn = reinterpret_cast<const void*>(sdq::mm4::matmul_pair_kernel<S, kF32>);
  static SmemLimit limit;
  if (const int e = limit.set(fn, static_cast<int>(Z::kSmem))) return e;
  const int64_t pairs = std::min<int64_t>(sms / 2, int64_t{p.tiles_a} * p.tiles_b);
  void* args[] = {&ma, &mb, &msa, &msb, &mo, &p};
  return launch(fn, static_cast<unsigned>(2 * pairs), sdq::mm4::kPairThreads, Z::kSmem, c.stream, args);
}

// CTAs that share the steps along k, in a cluster.  In quarters of a step (a step
// takes 0.3 us): the steps that are left to each, up to twice as long where two CTAs
// share a multiprocessor, and the exchange of the sums, a third of a quarter for each
// column and 16 more, twice that where eight CTAs of more than 32 columns exchange or
// where the next call's CTAs find few multiprocessors free to start on.  Only
// clusters that all fit at once: of four CTAs the device takes 33 (with one CTA a
// multiprocessor; 34 took 1.6 times as long), of eight with more than 32 columns
// fewer than 16.  us, E8M0 scales, with 1, 2, 4, 8 CTAs, the one chosen in brackets:
//       1 x  4096 x 7168   10.4   7.0  [5.0]  5.9    61 x 7168 x  4096  [7.6]  8.2  14.5  28.0
//       1 x  2048 x 1024    3.4   3.4  [2.9]  3.0    64 x 4096 x  7168  11.2   9.1  [8.7] 21.4
//       1 x 16384 x 7168   10.7 [10.4]               64 x 2048 x 14336  19.4  13.1  [9.2] 16.0
//      32 x  1024 x 7168   10.6   7.7   5.6  [4.4]  128 x 4096 x  7168  12.2 [11.3] 12.1  33.8
//      32 x 16384 x 1024   [3.7]  6.0               256 x 1024 x  4096  [8.5]  9.4   9.3  20.2
// Over 510 calls (1 to 256 rows, n 128 to 16384, k 512 to 14336) the one chosen takes
// 0.6 % more than the best of the four, 22 % at the worst (32 x 5632 x 14336).
int split_of(int cols, int64_t tiles, int64_t steps, int sms) {
  const bool wide = cols > sdq::mm4::kNarrow;
  int split = 1;
  int64_t best = 4 * steps;
  for (int s = 2; s <= 8 && s <= steps; s *= 2) {
    const int64_t ctas = tiles * s;
    const bool many = ctas > sms / 2;
    if (ctas * (s > 2 ? 10 : 9) > 9 * (wide ? sms : 2 * sms) || (wide && s == 8 && many)) break;
    const int64_t step = ctas <= sms ? 4 : s == 2 ? 7 : 8;
    const int64_t cost = (steps + s - 1) / s * step + (cols + 16) / 12 * (wide && (many || s == 8) ? 8 : 4);
    if (cost < best) {
      best = cost;
      split = s;
    }
  }
  return split;
}

// Few rows of a, or few tiles: clusters that share the steps along k.
template <Scales S>
int launch_strip(const Product& c, int sms) {
  using Z = sdq::mm4::StripShape<S>;
  sdq::mm4::Params p = {};
  p.sb = static_cast<const uint8_t*>(c.b_s);
  p.sa = static_cast<const uint8_t*>(c.a_s);
  p.ga = c.a_global;
  p.gb = c.b_global;
  p.out = static_cast<uint8_t*>(c.out);
  p.ld_out = c.ld_out;
  p.rows_a = c.m;
  p.rows_b = c.n;
  p.codes = static_cast<int32_t>(c.k);
  p.tiles_k = static_cast<int32_t>(tiles_of(c.k, c.format));
  p.cols = static_cast<int32_t>(std::min<int64_t>(128, up(c.m, 16)));
  p.tiles_b = static_cast<int32_t>((c.n + 127) / 128);
  p.stage = Z::stage(p.cols);
  p.out_f32 = c.format & SDQ_FMT_OUT_F32 ? 1 : 0;
  p.stall_step = c.stall_step;
  p.stall_rank = c.stall_rank;
  p.wait_limit_ns = c.wait_limit;
  if (const int e = sdq_internal::device_status_word(&p.status)) return e;
  CUtensorMap ma, mb;
  if (const int e = sdq_internal::make_code_map(&mb, c.b, c.k / 2, c.n, c.ld_b, 128)) return e;
  if (const int e = sdq_internal::make_code_map(&ma, c.a, c.k / 2, c.m, c.ld_a, p.cols)) return e;
  const void* fn = reinterpret_cast<const void*>(sdq::mm4::matmul_strip_kernel<S>);
  static SmemLimit limit;
  if (const int e = limit.set(fn, 210 * 1024)) return e;
  const int64_t tiles = p.tiles_b * ((c.m + p.cols - 1) / p.cols);
  const int64_t steps = (c.k + sdq::mm4::kStepCodes - 1) / sdq::mm4::kStepCodes;
  const int split = split_of(p.cols, tiles, steps, sms);
  p.stages = Z::stages(p.cols, split);
  p.share = Z::share(p.cols, split);
  for (int s = p.share; s > 1; s /= 2) ++p.share_log;
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage + Z::sums(p.cols, split);
  void* args[] = {&mb, &ma, &p};
  return launch(fn, static_cast<unsigned>(tiles * split), sdq::mm4::kThreads, smem, c.stream, args, split);
}

int launch_product(const Product& c) {
  int sms = 0;
  if (const int e = sdq_internal::sm_count(&sms)) return e;
  const bool e8m0 = c.format & SDQ_FMT_E8M0, f32 = c.format & SDQ_FMT_OUT_F32;
  // Tiles of 128 x 128 that the device takes at once: 128 columns a CTA keep more
  // multiprocessors busy than 256 x 256 outputs a pair (300 x 513 x 768: 4.5 us
  // instead of 7.1; 1024 x 1024 x 4096, 64 tiles: 8.6 and 9.2; 1024 x 2304 x 4096,
  // 144: 9.0 and 9.4).
  if (c.m <= 128 || (c.m + 127) / 128 * ((c.n + 127) / 128) <= sms)
    return e8m0 ? launch_strip<Scales::kE8M0>(c, sms) : launch_strip<Scales::kE4M3>(c, sms);
  if (f32) return e8m0 ? launch_pair<Scales::kE8M0, true>(c, sms) : launch_pair<Scales::kE4M3, true>(c, sms);
  return e8m0 ? launch_pair<Scales::kE8M0, false>(c, sms) : launch_pair<Scales::kE4M3, false>(c, sms);
}

}  // namespace

extern "C" {

int64_t sdq_fp4_scale_bytes(int64_t rows, int64_t k, uint32_t format) {
  if (rows < 0 || rows > SDQ_MAX_M || !length_ok(k) || !format_ok(format)) return 0;
  return (rows + 127) / 128 * tiles_of(k, format) * 512;
}

int sdq_validate_quantize_fp4(const void* x, int64_t ld_x, const void* q, int64_t ld_q, const void* s,
                              const void* q_t, int64_t ld_q_t, const void* s_t, const float* global_scale,
                              int64_t rows, int64_t channels, uint32_t format) {
  if (!format_ok(format)) return SDQ_ERR_FORMAT;
  if (rows < 0 || rows > SDQ_MAX_M || !length_ok(channels)) return SDQ_ERR_SHAPE;
  if ((rows + 127) / 128 * ((channels + 127) / 128) > INT32_MAX) return SDQ_ERR_SHAPE;
  if (rows == 0) return SDQ_OK;
  if (!x || (!q && !q_t) || (q && !s) || (q_t && !s_t)) return SDQ_ERR_NULL;
  if (ld_x < channels || ld_x > SDQ_MAX_LD) return SDQ_ERR_STRIDE;
  if (q && (ld_q < channels / 2 || ld_q > SDQ_MAX_LD)) return SDQ_ERR_STRIDE;
  if (q_t && (ld_q_t < up(rows, 32) / 2 || ld_q_t > SDQ_MAX_LD)) return SDQ_ERR_STRIDE;
  if (misaligned(x, 15) || (ld_x & 7) || misaligned(global_scale, 3)) return SDQ_ERR_ALIGN;
  if (q && (misaligned(q, 15) || (ld_q & 15) || misaligned(s, 15))) return SDQ_ERR_ALIGN;
  if (q_t && (misaligned(q_t, 15) || (ld_q_t & 15) || misaligned(s_t, 15))) return SDQ_ERR_ALIGN;
  return SDQ_OK;
}

int sdq_quantize_fp4(const void* x, int64_t ld_x, void* q, int64_t ld_q, void* s, void* q_t, int64_t ld_q_t, void* s_t,
                     const float* global_scale, int64_t rows, int64_t channels, uint32_t format, void* stream) {
  const int st = sdq_validate_quantize_fp4(x, ld_x, q, ld_q, s, q_t, ld_q_t, s_t, global_scale, rows, channels, format);
  if (st != SDQ_OK || rows == 0) return st;
  sdq::fp4::QuantParams p = {};
  p.x = static_cast<const uint8_t*>(x);
  p.q = static_cast<uint8_t*>(q);
  p.s = static_cast<uint8_t*>(s);
  p.qt = static_cast<uint8_t*>(q_t);
  p.st = static_cast<uint8_t*>(s_t);
  p.global = global_scale;
  p.rows = rows;
  p.ld_x = ld_x;
  p.ld_q = ld_q;
  p.ld_qt = ld_q_t;
  p.rows_padded = up(rows, 32);
  p.channels = static_cast<int32_t>(channels);
  p.tiles_k = static_cast<int32_t>(tiles_of(channels, format));
  p.tiles_m = tiles_of(p.rows_padded, format);
  p.grid_k = static_cast<int32_t>((channels + 127) / 128);
  const unsigned grid = static_cast<unsigned>((rows + 127) / 128 * p.grid_k);
  void* args[] = {&p};
  return launch(format & SDQ_FMT_E8M0 ? quantize_kernel<Scales::kE8M0>(q, q_t) : quantize_kernel<Scales::kE4M3>(q, q_t),
                grid, sdq::fp4::kThreads, 0, static_cast<cudaStream_t>(stream), args);
}

int sdq_validate_dequantize_fp4(const void* q, int64_t ld_q, const void* s, const float* global_scale, const void* out,
                                int64_t ld_out, int64_t rows, int64_t channels, uint32_t format) {
  if (!format_ok(format)) return SDQ_ERR_FORMAT;
  if (rows < 0 || rows > SDQ_MAX_M || !length_ok(channels)) return SDQ_ERR_SHAPE;
  if ((rows + 31) / 32 * ((channels + 255) / 256) > INT32_MAX) return SDQ_ERR_SHAPE;   // tiles of the grid
  if (rows == 0) return SDQ_OK;
  if (!q || !s || !out) return SDQ_ERR_NULL;
  if (ld_q < channels / 2 || ld_q > SDQ_MAX_LD || ld_out < channels || ld_out > SDQ_MAX_LD) return SDQ_ERR_STRIDE;
  if (misaligned(q, 15) || (ld_q & 15) || misaligned(s, 15) || misaligned(out, 15) || (ld_out & 7) ||
      misaligned(global_scale, 3))
    return SDQ_ERR_ALIGN;
  return SDQ_OK;
}

int sdq_dequantize_fp4(const void* q, int64_t ld_q, const void* s, const float* global_scale, void* out, int64_t ld_out,
                       int64_t rows, int64_t channels, uint32_t format, void* stream) {
  const int st = sdq_validate_dequantize_fp4(q, ld_q, s, global_scale, out, ld_out, rows, channels, format);
  if (st != SDQ_OK || rows == 0) return st;
  sdq::fp4::DequantParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.s = static_cast<const uint8_t*>(s);
  p.global = global_scale;
  p.out = static_cast<uint8_t*>(out);
  p.rows = rows;
  p.ld_q = ld_q;
  p.ld_out = ld_out;
  p.channels = static_cast<int32_t>(channels);
  p.tiles_k = static_cast<int32_t>(tiles_of(channels, format));
  constexpr int kRows = sdq::fp4::kThreads / 32 * sdq::fp4::kDequantRows;
  p.grid_k = static_cast<int32_t>((channels + sdq::fp4::kDequantCols - 1) / sdq::fp4::kDequantCols);
  void* args[] = {&p};
  return launch(format & SDQ_FMT_E8M0 ? reinterpret_cast<const void*>(sdq::fp4::dequantize_kernel<Scales::kE8M0>)
                                      : reinterpret_cast<const void*>(sdq::fp4::dequantize_kernel<Scales::kE4M3>),
                static_cast<unsigned>((rows + kRows - 1) / kRows * p.grid_k), sdq::fp4::kThreads, 0,
                static_cast<cudaStream_t>(stream), args);
}

int sdq_validate_matmul_fp4(const void* a, int64_t ld_a, const void* a_s, const float* a_global, const void* b,
                            int64_t ld_b, const void* b_s, const float* b_global, const void* out, int64_t ld_out,
                            int64_t m, int64_t n, int64_t k, uint32_t format) {
  if (!format_ok(format, SDQ_FMT_OUT_F32)) return SDQ_ERR_FORMAT;
  if (m < 0 || m > SDQ_MAX_M || n < 0 || n > SDQ_MAX_M || !length_ok(k)) return SDQ_ERR_SHAPE;
  if ((m + 127) / 128 * ((n + 127) / 128) > INT32_MAX) return SDQ_ERR_SHAPE;
  if (m == 0 || n == 0) return SDQ_OK;
  if (!a || !a_s || !b || !b_s || !out) return SDQ_ERR_NULL;
  if (ld_a < k / 2 || ld_a > SDQ_MAX_LD || ld_b < k / 2 || ld_b > SDQ_MAX_LD || ld_out < n || ld_out > SDQ_MAX_LD)
    return SDQ_ERR_STRIDE;
  if (misaligned(a, 15) || (ld_a & 15) || misaligned(b, 15) || (ld_b & 15) || misaligned(a_s, 15) ||
      misaligned(b_s, 15) || misaligned(a_global, 3) || misaligned(b_global, 3) ||
      misaligned(out, format & SDQ_FMT_OUT_F32 ? 3 : 1))
    return SDQ_ERR_ALIGN;
  return SDQ_OK;
}

int sdq_matmul_fp4(const void* a, int64_t ld_a, const void* a_s, const float* a_global, const void* b, int64_t ld_b,
                   const void* b_s, const float* b_global, void* out, int64_t ld_out, int64_t m, int64_t n, int64_t k,
                   uint32_t format, void* stream) {
  const int st = sdq_validate_matmul_fp4(a, ld_a, a_s, a_global, b, ld_b, b_s, b_global, out, ld_out, m, n, k, format);
  if (st != SDQ_OK || m == 0 || n == 0) return st;
  return launch_product({a, ld_a, a_s, a_global, b, ld_b, b_s, b_global, out, ld_out, m, n, k, format,
                         static_cast<cudaStream_t>(stream)});
}

int sdq_matmul_fp4_test_stall(const void* a, int64_t ld_a, const void* a_s, const void* b, int64_t ld_b, const void* b_s,
                              void* out, int64_t ld_out, int64_t m, int64_t n, int64_t k, uint32_t format, int32_t rank,
                              int32_t step, int64_t wait_limit_ns, void* stream) {
  const int st = sdq_validate_matmul_fp4(a, ld_a, a_s, nullptr, b, ld_b, b_s, nullptr, out, ld_out, m, n, k, format);
  if (st != SDQ_OK || m == 0 || n == 0) return st;
  if (rank < 0 || step < 0 || wait_limit_ns < 1000 || wait_limit_ns > 1000000000) return SDQ_ERR_SHAPE;
  return launch_product({a, ld_a, a_s, nullptr, b, ld_b, b_s, nullptr, out, ld_out, m, n, k, format,
                         static_cast<cudaStream_t>(stream), step, rank, static_cast<uint64_t>(wait_limit_ns)});
}

}  // extern "C"
