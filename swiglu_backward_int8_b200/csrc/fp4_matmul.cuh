// The product of two microscaled 4-bit operands, C = A B^T, on the tensor cores.
//
//   C[m, n] = alpha * sum_k (a[m, k] sa[m, k / G]) (b[n, k] sb[n, k / G])
//
// E2M1 codes two to a byte, G = 32 with E8M0 scales or G = 16 with E4M3
// scales, fp32 sums in tensor memory, alpha = the product of the two scales
// per tensor.  tcgen05.mma applies the block scales itself: it reads them
// from tensor memory, where tcgen05.cp puts the 512-byte scale tiles as they
// lie in memory (128 rows x 4 groups).
//
// This file: what both forms of the kernel share, and the form for few rows of A
// (matmul_strip_kernel).  The form for many is in fp4_matmul_pair.cuh.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "quant_common.cuh"

namespace sdq {
namespace mm4 {

using quant::Scales;

constexpr int kRows = 128;                  // lanes of the accumulator
constexpr int kStepBytes = 128;             // bytes of a row a stage holds: 256 codes
constexpr int kStepCodes = 2 * kStepBytes;
constexpr int kMmaCodes = 64;               // codes one tcgen05.mma takes along k
constexpr int kMmas = kStepCodes / kMmaCodes;
constexpr int kThreads = 192;               // a load warp, an mma warp, four epilogue warps

struct Params {
  const uint8_t* sb;       // scale tiles of B, whose rows are the accumulator's lanes
  const uint8_t* sa;       // of A, whose rows are its columns
  const float* ga;         // scales per tensor, or null
  const float* gb;
  uint8_t* out;            // [rows_a, rows_b]
  int64_t ld_out;          // elements
  int64_t rows_a, rows_b;
  int32_t codes;           // k
  int32_t tiles_k;         // scale tiles along k
  int32_t cols;            // columns a CTA computes: a multiple of 16, at most 128
  int32_t tiles_b;         // blocks of 128 rows of B
  int32_t stages, stage;   // the shared-memory ring
  int32_t share, share_log;   // columns that belong to a CTA of a cluster: a power of two
  int32_t out_f32;         // fp32 elements instead of bf16
  int32_t stall_step, stall_rank;   // the first load that this CTA of a cluster withholds (a test's; else -1)
  int* status;
  uint64_t wait_limit_ns;
};

// True in one lane of a converged warp.  A branch on it, unlike one on the lane's
// number, lets the compiler keep the descriptors of the tensor-core
// instructions in uniform registers; issuing them is what bound the kernels
// before (8192 x 14336 x 4096: 266 us, 179 with it).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// ---- tcgen05 -------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on the barrier once all tcgen05 work this thread has issued is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A scale tile from shared memory to 4 columns: 32 rows of 16 bytes, copied to
// each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <Scales S>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                    bool accumulate) {
  if (S == Scales::kE8M0)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// 32 columns of the warp's 32 lanes; the registers are valid after load_wait().
__device__ __forceinline__ void load_sums32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void load_sums16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory descriptors (start address, strides in units of 16 bytes,
// version 1): K-major rows of 128 swizzled bytes, eight rows every 1024; and
// the scale tiles, unswizzled, eight rows of 16 bytes every 128.
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (8ull << 32) | (1ull << 46);
}

// Instruction descriptor of the block-scaled 4-bit kinds: E2M1 operands
// (format 1 at bits 7 and 10), n / 8 at bit 17, E8M0 scales at bit 23,
// m / 128 at bit 27; the scale's first byte in its column word goes to bits 4
// (B) and 29 (A).
template <Scales S>
__device__ __forceinline__ uint32_t instruction(int m, int n, uint32_t scale_byte) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n / 8) << 17) | (S == Scales::kE8M0 ? 1u << 23 : 0u) |
         (static_cast<uint32_t>(m / 128) << 27) | (scale_byte << 4) | (scale_byte << 29);
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// ---- clusters -----------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, for the whole cluster, of this shared-memory address in CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_cluster4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float4 load_shared4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// ---- waits ----------------------------------------------------------------------

struct Sync {
  int* status;         // the device status word
  volatile int* abort; // shared: set by the first wait that runs out
  uint64_t limit_ns;
};

// Waits for the barrier's phase, no longer than the limit; false once any
// wait of the CTA has run out.
__device__ __forceinline__ bool wait(const Sync& y, uint32_t bar, uint32_t parity) {
  // (a try_wait suspends the thread for a while by itself; the timer, slow to
  // read, comes in only once several have run out)
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*y.abort) return false;
    if (globaltimer_ns() - t0 > y.limit_ns) {
      *y.abort = 1;
      atomicOr(y.status, 1);
      return false;
    }
  }
  return true;
}

// What a CTA has in flight when a wait has run out (copies into its shared memory,
// signals to its barriers) lands before it leaves: waited for, in all no longer
// than a second, however short the waits' own limit.
struct Drain {
  static constexpr uint64_t kLimitNs = 1000000000;
  const uint64_t t0 = globaltimer_ns();
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) const {
    const uint64_t used = globaltimer_ns() - t0;
    mbar_wait(bar, parity, used < kLimitNs ? kLimitNs - used : 0);
  }
};

// Whether all lanes say so: each decides by itself whether its wait has run out, and
// what follows takes the warp together (tcgen05.ld, a barrier of the cluster).
__device__ __forceinline__ bool all_lanes(bool v) { return __all_sync(0xffffffffu, v); }

// ---- the scales per tensor ------------------------------------------------------

// What the sums are multiplied by: the product of the two scales per tensor, or,
// where that leaves fp32's normal range, first the larger and then the smaller (a
// sum times both can be well inside: 1e-25 and 1e-18 with sums of 1e9).
struct Alpha {
  float pre = 1.0f, last = 1.0f;
  __device__ __forceinline__ void set(const float* ga, const float* gb) {
    const float a = ga ? *ga : 1.0f, b = gb ? *gb : 1.0f;
    last = a * b;
    if (!(fabsf(last) >= 1.17549435e-38f && fabsf(last) <= 3.40282347e38f) && a == a && b == b) {
      pre = fmaxf(a, b);
      last = fminf(a, b);
    }
  }
  __device__ __forceinline__ float of(float sum) const { return sum * pre * last; }
};

// ---- the kernel for few rows of A -----------------------------------------------------
//
// Reading B bounds it, and below some 8 MB the launch and the latencies in a row
// (wait for the kernel before, first load, exchange, store: 5 us).  B's rows are the accumulator's lanes, 128 a CTA, and A's its
// columns, so an instruction is no wider than A needs.  The CTAs of a cluster take
// the steps along k in turn, where that is worth the exchange (split_of); each sends its sums to the CTA that a column belongs to (column c to rank
// c / share), which adds them up in the order of the ranks: the result does not
// depend on timing.  (Sending takes one barrier of the cluster; reading the
// others' sums took two, and a latency a number.)  Up to 32 columns two CTAs fit a
// multiprocessor: a kernel's set-up is under way while the one before it still
// runs.  1 x 4096 x 7168: 5.0 us (10.4 with one CTA for all of k), of 2.5 that its
// bytes take; 61 x 7168 x 4096: 7.8 us.

// Where a lane's next output goes: its column of `out`, a row further each time.
struct Column {
  uint8_t* at;
  int64_t step;
  int f32;
  __device__ __forceinline__ Column(const Params& p, int64_t row, int64_t col)
      : at(p.out + (row * p.ld_out + col) * (p.out_f32 ? 4 : 2)), step(p.ld_out * (p.out_f32 ? 4 : 2)), f32(p.out_f32) {}
  __device__ __forceinline__ void put(float v) {
    if (f32)
      *reinterpret_cast<float*>(at) = v;
    else
      *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    at += step;
  }
};

constexpr int kMaxStages = 8;
constexpr int kNarrow = 32;   // columns up to which two CTAs share a multiprocessor

template <Scales S>
struct StripShape {
  static constexpr int kScaleTiles = S == Scales::kE8M0 ? 2 : 4;   // scale tiles a stage holds of either side
  static constexpr int kScale = kScaleTiles * 512;
  static constexpr int kCodesB = kRows * kStepBytes;
  static constexpr int kColsScale = 2 * kScaleTiles * 4;           // tensor memory: a set of both sides' scales
  static constexpr int kCols = 256;                                // 128 sums and two sets of scales used in turn
  static_assert(128 + 2 * kColsScale <= kCols, "the sums and the scales fit");
  static int stage(int cols) { return kCodesB + cols * kStepBytes + 2 * kScale; }   // a multiple of 1024
  // Columns that belong to a CTA: a power of two, at least the four of a vector.
  static int share(int cols, int split) {
    int s = 4;
    while (s * split < cols) s *= 2;
    return s;
  }
  static int sums(int cols, int split) { return split > 1 ? split * share(cols, split) * kRows * 4 : 0; }
  static int stages(int cols, int split) {
    const int n = ((cols <= kNarrow ? 108 : 208) * 1024 - sums(cols, split)) / stage(cols);
    return n > kMaxStages ? kMaxStages : n;
  }
};

template <Scales S>
__global__ void __launch_bounds__(kThreads, 2)
    matmul_strip_kernel(const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap ma, const Params p) {
  using Z = StripShape<S>;
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[2 * kMaxStages + 1];
  __shared__ uint32_t tmem_addr;
  __shared__ int abort_flag, issued_flag;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;   // the same offset in every CTA of the cluster
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages, done = empty + 8 * kMaxStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
  const int tile = blockIdx.x / ranks;
  const int tile_a = tile / p.tiles_b, tile_b = tile - tile_a * p.tiles_b;
  const int64_t b0 = static_cast<int64_t>(tile_b) * kRows, a0 = static_cast<int64_t>(tile_a) * p.cols;
  const int steps_all = (p.codes + kStepCodes - 1) / kStepCodes;
  const int steps = (steps_all - rank + ranks - 1) / ranks;   // steps rank, rank + ranks, ...: at least one
  if (threadIdx.x == 0) {
    prefetch_tensormap(&mb);
    prefetch_tensormap(&ma);
    for (int i = 0; i < 2 * kMaxStages + 1; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
    abort_flag = 0;
    issued_flag = 0;
  }
  if (warp == 0 && elect_one())   // into L2 only: changes no value that is read after the wait below
    for (int i = 0; i < steps && i < p.stages; ++i)
      tma_prefetch_l2_2d(&mb, (rank + i * ranks) * kStepBytes, static_cast<int32_t>(b0));
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_addr), Z::kCols);
    tmem_relinquish();
    fence_before();
  }
  __syncthreads();
  if (ranks > 1) cluster_arrive();   // waited for before the first store into another CTA: all have started
  fence_after();
  grid_dependency_wait();     // operands may come from the previous kernel in the stream
  grid_launch_dependents();   // after the allocation: a later kernel's cannot come first
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&tmem_addr);
  const Sync sync = {p.status, &abort_flag, p.wait_limit_ns};
  const uint32_t parts = ring + p.stages * p.stage;   // the sums that this CTA receives
  // The sums of a rank's row lie in vectors of four, swizzled by the row so that
  // neither the senders' lanes nor the reader's meet in a bank.
  const int vecs = p.share >> 2, mask = vecs < 8 ? vecs - 1 : 7, shift = vecs < 2 ? 3 : vecs < 4 ? 2 : vecs < 8 ? 1 : 0;
  auto slot = [&](int from, int row, int vec) {
    return parts + static_cast<uint32_t>(((from * kRows + row) * vecs + (vec ^ ((row >> shift) & mask))) << 4);
  };

  Alpha alpha;
  if (warp == 0) {
    if (elect_one()) {
      for (int i = 0; i < steps; ++i) {
        const int st = i % p.stages, step = rank + i * ranks;
        if (i == p.stall_step && rank == p.stall_rank) break;
        if (i >= p.stages && !wait(sync, empty + 8 * st, ((i / p.stages) - 1) & 1)) break;
        const uint32_t buf = ring + st * p.stage, bar = full + 8 * st;
        const int k_tile = step * Z::kScaleTiles;
        const int tiles = min(Z::kScaleTiles, p.tiles_k - k_tile);
        mbar_arrive_expect_tx(bar, Z::kCodesB + p.cols * kStepBytes + 2 * tiles * 512);
        tma_load(buf, &mb, bar, step * kStepBytes, static_cast<int32_t>(b0));
        tma_load(buf + Z::kCodesB, &ma, bar, step * kStepBytes, static_cast<int32_t>(a0));
        const uint32_t sc = buf + Z::kCodesB + p.cols * kStepBytes;
        bulk_load(sc, p.sb + (static_cast<int64_t>(tile_b) * p.tiles_k + k_tile) * 512, tiles * 512, bar);
        bulk_load(sc + Z::kScale, p.sa + ((a0 >> 7) * p.tiles_k + k_tile) * 512, tiles * 512, bar);
        issued_flag = i + 1;
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t id0 = instruction<S>(kRows, p.cols, 0), id1 = S == Scales::kE8M0 ? instruction<S>(kRows, p.cols, 2) : id0;
      for (int i = 0; i < steps; ++i) {
        const int st = i % p.stages, step = rank + i * ranks;
        if (!wait(sync, full + 8 * st, (i / p.stages) & 1)) break;
        fence_after();
        const uint32_t buf = ring + st * p.stage;
        const uint32_t tb = tmem + 128 + (i & 1) * Z::kColsScale, ta = tb + Z::kScaleTiles * 4;
        const uint64_t ds = desc_scales(buf + Z::kCodesB + p.cols * kStepBytes);
#pragma unroll
        for (int j = 0; j < Z::kScaleTiles; ++j) {
          copy_scales(tb + 4 * j, ds + 32 * j);
          copy_scales(ta + 4 * j, ds + (Z::kScale >> 4) + 32 * j);
        }
        const uint64_t db = desc_codes(buf), da = desc_codes(buf + Z::kCodesB);
        const int mmas = min(kMmas, (p.codes - step * kStepCodes + kMmaCodes - 1) / kMmaCodes);
#pragma unroll
        for (int j = 0; j < kMmas; ++j) {
          constexpr int kPerTile = S == Scales::kE8M0 ? 2 : 1;   // products a scale tile lasts
          if (j < mmas)
            mma<S>(tmem, db + 2 * j, da + 2 * j, (j & 1) ? id1 : id0, tb + 4 * (j / kPerTile), ta + 4 * (j / kPerTile),
                   i > 0 || j > 0);
        }
        commit(empty + 8 * st);
      }
      commit(done);
      Drain().wait(done, 0);   // nothing of the tensor cores is in flight when the CTA frees its memory
    }
  } else {
    alpha.set(p.ga, p.gb);   // while the sums are computed
    const bool ok = all_lanes(wait(sync, done, 0) && !*sync.abort);
    fence_after();
    const int quarter = warp & 3;   // the lanes a warp may read
    const int row = quarter * 32 + lane;
    const int cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.rows_a - a0));
    if (ranks > 1) {
      __syncwarp();
      cluster_wait();
    }
    Column mine(p, a0, b0 + row);
    for (int c = 0; ok && c < cols; c += 16) {
      uint32_t r[16];
      load_sums16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
      load_wait();
      if (ranks > 1) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          store_cluster4(at_rank(slot(rank, row, ((c + e) & (p.share - 1)) >> 2), (c + e) >> p.share_log), &r[e]);
      } else if (b0 + row < p.rows_b) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c + e < cols) mine.put(alpha.of(__uint_as_float(r[e])));
      }
    }
    fence_before();
  }
  if (warp < 2 && ranks > 1) {   // the barriers count every thread
    __syncwarp();
    cluster_wait();
  }
  __syncthreads();
  __syncwarp();
  // Tensor memory goes back before the CTA waits for others: a CTA of theirs may
  // be waiting for it, behind another kernel that waits for this one.
  if (warp == 1) {
    fence_after();
    tmem_free(tmem, Z::kCols);
  }
  if (ranks > 1) {   // (after a wait that ran out the sums are of no use, as the status says)
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    const int row = (warp & 3) * 32 + lane;
    if (warp >= 2 && b0 + row < p.rows_b) {
      const int cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.rows_a - a0));
      const int first = rank * p.share, last = min(first + p.share, cols);
      Column out(p, a0 + first, b0 + row);
      for (int c = first; c < last; c += 4) {
        float4 v = load_shared4(slot(0, row, (c - first) >> 2));
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          if (r < ranks) {
            const float4 u = load_shared4(slot(r, row, (c - first) >> 2));
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
          }
        }
        const float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < last) out.put(alpha.of(s[e]));
      }
    }
  }
  if (threadIdx.x == 0 && abort_flag) {   // copies still in flight write this CTA's shared memory
    const Drain drain;
    for (int i = max(0, issued_flag - p.stages); i < issued_flag; ++i)
      drain.wait(full + 8 * (i % p.stages), (i / p.stages) & 1);
  }
}

}  // namespace mm4
}  // namespace sdq
