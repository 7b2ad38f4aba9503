// C ABI of the quantizing RMS norm and its backward (declared in
// include/sdq.h): argument validation, the choice of the variant, the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_kernel.cuh"
#include "sdq.h"
#include "sdq_internal.h"

namespace {

using sdq::norm::BwdParams;
using sdq::norm::Params;
using sdq::quant::Codes;
using sdq::quant::Scales;

enum class Variant { kFew, kMany, kLong };

template <Codes C, Scales S>
const void* kernel_of(Variant v) {
  return v == Variant::kFew    ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_quant_kernel<C, S>)
         : v == Variant::kMany ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_quant_rows_kernel<C, S>)
                               : reinterpret_cast<const void*>(sdq::norm::rmsnorm_quant_long_kernel<C, S>);
}

const void* kernel_for(uint32_t format, Variant v) {
  const bool e8 = format & SDQ_FMT_E8M0;
  if (format & SDQ_FMT_E2M1)
    return e8 ? kernel_of<Codes::kE2M1, Scales::kE8M0>(v) : kernel_of<Codes::kE2M1, Scales::kE4M3>(v);
  if (format & SDQ_FMT_E4M3)
    return e8 ? kernel_of<Codes::kE4M3, Scales::kE8M0>(v) : kernel_of<Codes::kE4M3, Scales::kF32>(v);
  return e8 ? kernel_of<Codes::kInt8, Scales::kE8M0>(v) : kernel_of<Codes::kInt8, Scales::kF32>(v);
}

constexpr uint32_t kFormatBits = SDQ_FMT_E4M3 | SDQ_FMT_E8M0 | SDQ_FMT_E2M1 | SDQ_FMT_SCALE_E4M3 | SDQ_FMT_WEIGHT_F32;
// Values up to which the backward is one kernel that reads grad_y and h twice
// (from L2), where the rows are few besides: 517 x 7168 9.2 us instead of 11.3,
// but 1000 x 512 8.5 instead of 4.8.
constexpr int64_t kFewValues = int64_t{1} << 22;
constexpr int64_t kMaxParts = 592;   // rows of partial weight gradients a backward keeps: four a multiprocessor

// The codes' and scales' formats go together: 8-bit codes with fp32 or E8M0
// scales, E2M1 codes with E8M0 or E4M3 scales.
bool format_ok(uint32_t f) {
  if (f & ~kFormatBits) return false;
  const bool e2m1 = f & SDQ_FMT_E2M1, e4m3 = f & SDQ_FMT_E4M3, e8 = f & SDQ_FMT_E8M0, s4 = f & SDQ_FMT_SCALE_E4M3;
  if (e2m1 && e4m3) return false;
  return e2m1 ? e8 != s4 : !s4;
}

bool group_ok(int32_t g, uint32_t f) {
  if (f & SDQ_FMT_E2M1) return g == (f & SDQ_FMT_E8M0 ? 32 : 16);
  return g == 0 || g == 32 || g == 64 || g == 128 || g == 256;
}

bool misaligned(const void* p, uintptr_t mask) { return reinterpret_cast<uintptr_t>(p) & mask; }

// A bf16 array of rows: unset, or its stride and alignment right.
int check_rows(const void* p, int64_t ld, int64_t channels) {
  if (ld < channels || ld > SDQ_MAX_LD_NORM) return SDQ_ERR_STRIDE;
  return misaligned(p, 15) || (ld & 7) ? SDQ_ERR_ALIGN : SDQ_OK;
}

int launch(const void* kernel, dim3 grid, dim3 block, cudaStream_t stream, void** args, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  return e == cudaSuccess ? SDQ_OK : sdq_internal::cuda_fail(e);
}

// Whether two bf16 arrays of rows share memory (or lie in each other's gaps).
bool overlap(const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t rows, int64_t channels) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  const uintptr_t na = 2 * static_cast<uintptr_t>((rows - 1) * ld_a + channels);
  const uintptr_t nb = 2 * static_cast<uintptr_t>((rows - 1) * ld_b + channels);
  return pa < pb + nb && pb < pa + na;
}

int round_up(int v, int m) { return (v + m - 1) / m * m; }

// Threads of a row of `vecs` vectors where several rows share a CTA: 4, 8 or 16
// lanes, or whole warps.
int threads_of(int vecs) { return vecs <= 4 ? 4 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : round_up(vecs, 32); }

// CTAs of `threads` threads with `regs` registers each that a multiprocessor
// holds: each quarter of it has 16384 registers.  (A grid that leaves room for more
// is the worse also because the next kernel's CTAs, which wait there, then spread
// unevenly: 16384 x 1408, three warps a row, ten CTAs: 25.1 us a call in a row of
// them, with eight 30.3.)
int ctas_per_sm(int threads, int regs) {
  const int warps = 4 * (16384 / (32 * regs));
  return std::max(1, std::min(warps / (threads / 32), 2048 / threads));
}

}  // namespace

extern "C" {

int sdq_validate_rmsnorm_quant(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                               const void* weight, const void* h, int64_t ld_h, const void* q, int64_t ld_q,
                               const void* s, int64_t ld_s, const void* y, int64_t ld_y, const float* rstd,
                               const float* global_scale, int64_t rows, int64_t channels, int32_t group_size,
                               uint32_t format) {
  if (!format_ok(format)) return SDQ_ERR_FORMAT;
  if (!group_ok(group_size, format)) return SDQ_ERR_GROUP;
  const bool e2m1 = format & SDQ_FMT_E2M1;
  if (rows < 0 || rows > SDQ_MAX_M || channels < 1 || channels > SDQ_MAX_K ||
      channels % (e2m1 ? SDQ_FP4_K_MULTIPLE : SDQ_K_MULTIPLE) != 0)
    return SDQ_ERR_SHAPE;
  if (rows == 0) return SDQ_OK;
  if (!x || !weight || !q || !s || (residual && !h)) return SDQ_ERR_NULL;
  int st = check_rows(x, ld_x, channels);
  if (st == SDQ_OK && residual) st = check_rows(residual, ld_residual, channels);
  if (st == SDQ_OK && residual) st = check_rows(h, ld_h, channels);
  if (st == SDQ_OK && y) st = check_rows(y, ld_y, channels);
  if (st != SDQ_OK) return st;
  const int64_t qbytes = e2m1 ? channels / 2 : channels;
  if (ld_q < qbytes || ld_q > SDQ_MAX_LD_NORM) return SDQ_ERR_STRIDE;
  if (!e2m1) {
    const int64_t g = group_size ? group_size : channels;
    if (ld_s < (channels + g - 1) / g || ld_s > SDQ_MAX_LD_NORM) return SDQ_ERR_STRIDE;
  }
  if (misaligned(q, 15) || (ld_q & 15) || misaligned(weight, 15) || misaligned(rstd, 3) || misaligned(global_scale, 3))
    return SDQ_ERR_ALIGN;
  if (misaligned(s, e2m1 ? 15 : (format & SDQ_FMT_E8M0) ? 0 : 3)) return SDQ_ERR_ALIGN;
  return SDQ_OK;
}

int sdq_rmsnorm_quant(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                      void* h, int64_t ld_h, void* q, int64_t ld_q, void* s, int64_t ld_s, void* y, int64_t ld_y,
                      float* rstd, const float* global_scale, int64_t rows, int64_t channels, int32_t group_size,
                      uint32_t format, float eps, void* stream) {
  const int st = sdq_validate_rmsnorm_quant(x, ld_x, residual, ld_residual, weight, h, ld_h, q, ld_q, s, ld_s, y, ld_y,
                                            rstd, global_scale, rows, channels, group_size, format);
  if (st != SDQ_OK || rows == 0) return st;
  int sms = 0;
  if (const int e = sdq_internal::sm_count(&sms)) return e;
  const int groups = static_cast<int>(group_size ? (channels + group_size - 1) / group_size : 1);
  Params p = {};
  p.x = static_cast<const uint8_t*>(x);
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint8_t*>(weight);
  p.h = static_cast<uint8_t*>(h);
  p.q = static_cast<uint8_t*>(q);
  p.s = static_cast<uint8_t*>(s);
  p.y = static_cast<uint8_t*>(y);
  p.rstd = rstd;
  p.global = global_scale;
  p.rows = rows;
  p.ld_x = static_cast<uint32_t>(ld_x);
  p.ld_residual = static_cast<uint32_t>(ld_residual);
  p.ld_h = static_cast<uint32_t>(ld_h);
  p.ld_q = static_cast<uint32_t>(ld_q);
  p.ld_s = static_cast<uint32_t>(ld_s);
  p.ld_y = static_cast<uint32_t>(ld_y);
  p.channels = static_cast<int32_t>(channels);
  p.group = group_size;
  p.groups = groups;
  p.tiles_k = (groups + 3) / 4;
  p.weight_f32 = format & SDQ_FMT_WEIGHT_F32 ? 1 : 0;
  p.eps = eps;
  p.inv_channels = 1.0f / static_cast<float>(channels);
  const int vecs = static_cast<int>(channels / sdq::norm::kVec);
  // A vector a thread.  Few rows: each its own CTA.  Many: a persistent grid,
  // the next row loaded ahead.  Rows that no CTA holds: read again.
  const Variant v = vecs > sdq::norm::kMaxThreads ? Variant::kLong : rows <= sms ? Variant::kFew : Variant::kMany;
  int row_threads = v == Variant::kLong ? sdq::norm::kMaxThreads : v == Variant::kMany ? threads_of(vecs) : round_up(vecs, 32);
  const int rows_cta = v == Variant::kMany ? std::max(1, 128 / row_threads) : 1;
  int64_t grid = (rows + rows_cta - 1) / rows_cta;
  if (v == Variant::kMany)
    grid = std::min<int64_t>(grid, int64_t{sms} * ctas_per_sm(row_threads * rows_cta, sdq::norm::kAheadRegs));
  void* args[] = {&p, &row_threads};
  return launch(kernel_for(format, v), dim3(static_cast<unsigned>(grid)), dim3(row_threads * rows_cta),
                static_cast<cudaStream_t>(stream), args);
}

size_t sdq_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t channels) {
  if (rows < 0 || rows > SDQ_MAX_M || channels < 1 || channels > SDQ_MAX_K || channels % SDQ_K_MULTIPLE != 0) return 0;
  return static_cast<size_t>(std::max<int64_t>(1, std::min(rows, kMaxParts)) * channels * 4);
}

int sdq_validate_rmsnorm_backward(const void* grad_y, int64_t ld_grad_y, const void* h, int64_t ld_h,
                                  const void* weight, const float* rstd, const void* grad_h, int64_t ld_grad_h,
                                  const void* grad_x, int64_t ld_grad_x, const float* grad_weight, int64_t rows,
                                  int64_t channels, uint32_t format, const void* workspace, size_t workspace_bytes) {
  if (format & ~SDQ_FMT_WEIGHT_F32) return SDQ_ERR_FORMAT;
  const size_t need = sdq_rmsnorm_backward_workspace_bytes(rows, channels);
  if (need == 0) return SDQ_ERR_SHAPE;
  if (!grad_weight || (rows > 0 && (!grad_y || !h || !weight || !rstd || !grad_x || !workspace))) return SDQ_ERR_NULL;
  if (misaligned(grad_weight, 3)) return SDQ_ERR_ALIGN;
  if (rows == 0) return SDQ_OK;
  int st = check_rows(grad_y, ld_grad_y, channels);
  if (st == SDQ_OK) st = check_rows(h, ld_h, channels);
  if (st == SDQ_OK && grad_h) st = check_rows(grad_h, ld_grad_h, channels);
  if (st == SDQ_OK) st = check_rows(grad_x, ld_grad_x, channels);
  if (st != SDQ_OK) return st;
  if (misaligned(weight, 15) || misaligned(rstd, 3)) return SDQ_ERR_ALIGN;
  if (workspace_bytes < need || misaligned(workspace, 15)) return SDQ_ERR_WORKSPACE;
  return SDQ_OK;
}

int sdq_rmsnorm_backward(const void* grad_y, int64_t ld_grad_y, const void* h, int64_t ld_h, const void* weight,
                         const float* rstd, const void* grad_h, int64_t ld_grad_h, void* grad_x, int64_t ld_grad_x,
                         float* grad_weight, int64_t rows, int64_t channels, uint32_t format, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const int st = sdq_validate_rmsnorm_backward(grad_y, ld_grad_y, h, ld_h, weight, rstd, grad_h, ld_grad_h, grad_x,
                                               ld_grad_x, grad_weight, rows, channels, format, workspace,
                                               workspace_bytes);
  if (st != SDQ_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // an empty sum
    const cudaError_t e = cudaMemsetAsync(grad_weight, 0, 4 * static_cast<size_t>(channels), s);
    return e == cudaSuccess ? SDQ_OK : sdq_internal::cuda_fail(e);
  }
  int sms = 0;
  if (const int e = sdq_internal::sm_count(&sms)) return e;
  BwdParams p = {};
  p.gy = static_cast<const uint8_t*>(grad_y);
  p.h = static_cast<const uint8_t*>(h);
  p.weight = static_cast<const uint8_t*>(weight);
  p.rstd = rstd;
  p.gh = static_cast<const uint8_t*>(grad_h);
  p.gx = static_cast<uint8_t*>(grad_x);
  p.gw = grad_weight;
  p.part = static_cast<float*>(workspace);
  p.rows = rows;
  p.ld_gy = static_cast<uint32_t>(ld_grad_y);
  p.ld_h = static_cast<uint32_t>(ld_h);
  p.ld_gh = static_cast<uint32_t>(ld_grad_h);
  p.ld_gx = static_cast<uint32_t>(ld_grad_x);
  p.channels = static_cast<int32_t>(channels);
  p.inv_channels = 1.0f / static_cast<float>(channels);
  p.weight_f32 = format & SDQ_FMT_WEIGHT_F32 ? 1 : 0;
  const int vecs = static_cast<int>((channels + 7) / 8);
  const int kv_few = vecs <= 512 ? 1 : 2;
  int threads_few = threads_of((vecs + kv_few - 1) / kv_few);
  // CTAs of up to 1024 threads for short rows (900 x 2048: 6.7 us, 8.8 with 512
  // threads; 512 x 4096: 6.4 and 8.5 with two rows a CTA): the weight's gradient
  // takes threads / 8 rows at a time, and is what takes longest where rows are
  // short.  More of them are left to the kernel below (2000 x 256: 6.8 us, 4.7 there).
  // (Weight's CTAs read grad_y and h while others write grad_x: not where that is
  // written over them.)
  const int rows_few = vecs <= 384 ? std::max(1, 1024 / threads_few) : 1;
  const bool over = overlap(grad_x, ld_grad_x, grad_y, ld_grad_y, rows, channels) ||
                    overlap(grad_x, ld_grad_x, h, ld_h, rows, channels);
  if (!over && vecs <= 2 * sdq::norm::kMaxThreads && rows * channels <= kFewValues && rows <= 600 + 8 * vecs) {
    int weight_ctas = static_cast<int>((channels + sdq::norm::kWeightCols - 1) / sdq::norm::kWeightCols);
    void* args[] = {&p, &threads_few, &weight_ctas};
    return launch(kv_few == 1 ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_few_kernel<1>)
                          : reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_few_kernel<2>),
                  dim3(static_cast<unsigned>(weight_ctas + (rows + rows_few - 1) / rows_few)),
                  dim3(threads_few * rows_few), s, args);
  }
  // Vectors a thread: two, or four where two leave a multiprocessor one CTA (8192 x
  // 8192: 103 us with two, 99 with four; 16384 x 4096: 92 and 96).  Rows a CTA:
  // several short ones.
  const int kv = vecs <= 16 ? 1 : vecs <= 768 ? 2 : vecs <= 2048 ? 4 : 0;
  const bool several = vecs <= 256;
  int row_threads = several ? threads_of((vecs + kv - 1) / kv) : kv ? round_up((vecs + kv - 1) / kv, 32) : sdq::norm::kMaxThreads;
  const int rows_cta = several ? std::max(1, 256 / row_threads) : 1;
  const int threads = row_threads * rows_cta;
  const int per_sm = kv ? std::min(4, ctas_per_sm(threads, sdq::norm::backward_regs(kv))) : 1;
  p.parts = static_cast<int32_t>(
      std::min<int64_t>((rows + rows_cta - 1) / rows_cta, std::min<int64_t>(kMaxParts, int64_t{sms} * per_sm)));
  const void* k = kv == 0   ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_long_kernel)
                  : kv == 1 ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_kernel<1, true>)
                  : several ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_kernel<2, true>)
                  : kv == 2 ? reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_kernel<2, false>)
                            : reinterpret_cast<const void*>(sdq::norm::rmsnorm_backward_kernel<4, false>);
  // at most 256 / row_threads rows of 16 row_threads channels: 16 KB
  const size_t smem = rows_cta > 1 ? static_cast<size_t>(rows_cta) * channels * 4 : 0;
  void* args[] = {&p, &row_threads};
  if (const int e = launch(k, dim3(p.parts), dim3(threads), s, args, smem)) return e;
  const float* part = p.part;
  void* args2[] = {&part, &p.gw, &p.parts, &p.channels};
  return launch(reinterpret_cast<const void*>(sdq::norm::grad_weight_kernel),
                dim3(static_cast<unsigned>((channels + 31) / 32)), dim3(1024), s, args2);
}

}  // extern "C"
