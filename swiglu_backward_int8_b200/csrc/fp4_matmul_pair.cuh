// The large form of the product C = A B^T of two microscaled 4-bit operands
// (fp4_matmul.cuh): two multiprocessors share a tile of 256 x 256 outputs
// (tcgen05.mma with cta_group::2), and a persistent grid of such pairs walks
// the tiles, a tile's sums being read out while the next one is computed.
//
// Why pairs: a CTA's half of the tile needs 128 rows of A and only its half of
// the rows of B in its own shared memory, so an instruction reads 64 bytes a
// cycle of it at the tensor cores' 4-bit rate, where a single CTA's 128 x 256
// tile would read 96 and be refilled at 100 more.
//
// Tensor memory: two accumulators of 256 columns and two sets of scales do not
// fit, so the accumulators share columns: the second starts where the first
// still has some to go, and the epilogue of either reads those first and gives
// them back.
//
// What bounds it: filling shared memory from L2.  A stage is 35 KB (38 with E4M3
// scales) a multiprocessor, and 82 GB/s each (12 TB/s in all) is what the loads
// reach with the products taken out: 170 of the 175 us of 8192 x 14336 x 4096 at
// full clock (5.5 PFLOP/s; with E4M3 scales 185).  Back to back for a second the
// power limit lowers the clock: 208 us (4.6 PFLOP/s).
#pragma once

#include "fp4_matmul.cuh"

namespace sdq {
namespace mm4 {

constexpr int kEpilogueWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpilogueWarps;   // a load warp, an mma warp, the epilogue's

constexpr int kN = 256;   // columns of a tile

template <Scales S>
struct PairShape {
  static constexpr int kScaleTiles = S == Scales::kE8M0 ? 2 : 4;   // a stage's scale tiles per 128 rows
  static constexpr int kBlocksB = kN / 128;
  static constexpr int kCodesA = kRows * kStepBytes;
  static constexpr int kCodesB = kN / 2 * kStepBytes;
  static constexpr int kScaleA = kScaleTiles * 512;
  static constexpr int kScaleB = kBlocksB * kScaleTiles * 512;
  static constexpr int kStage = kCodesA + kCodesB + kScaleA + kScaleB;
  static constexpr int kBoxes = kEpilogueWarps * 32 * 128;   // a box of output an epilogue warp
  static constexpr int kStages = (226 * 1024 - 1024 - kBoxes) / kStage > 8 ? 8 : (226 * 1024 - 1024 - kBoxes) / kStage;
  static constexpr int kColsScaleA = kScaleTiles * 4;
  static constexpr int kColsScale = kColsScaleA + kScaleTiles * 4 * kBlocksB;
  static constexpr int kScaleCol = 512 - 2 * kColsScale;
  static constexpr int kAcc1 = (kScaleCol - kN) / 64 * 64;   // the second accumulator's first column
  static constexpr int kShared = kN - kAcc1;                                // columns both accumulators use
  static constexpr size_t kSmem = 1024 + kStages * static_cast<size_t>(kStage) + kBoxes;
  static_assert(kStage % 1024 == 0, "the swizzled boxes start on 1024 bytes");
  static_assert(kAcc1 >= 0 && kAcc1 % 64 == 0 && kShared % 64 == 0 && kShared > 0 && kShared <= 128,
                "whole pieces of 64 columns, those that are shared the first of a warp");
};

struct PairParams {
  const float* ga;
  const float* gb;
  uint8_t* out;
  int64_t ld_out;
  int64_t rows_a, rows_b;
  int32_t codes;
  int32_t tiles_a, tiles_b;
  int32_t vec;             // the output's rows start on 16 bytes: bulk stores
  int32_t stall_step, stall_rank;   // the first load that this CTA of a pair withholds (a test's; else -1)
  int* status;
  uint64_t wait_limit_ns;
};

// ---- pairs ------------------------------------------------------------------------

__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// A box into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t c0,
                                              int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(cluster_bar)
      : "memory");
}
// Counts bytes on a barrier of this CTA as landed that will not come.
__device__ __forceinline__ void complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t cluster_bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <Scales S>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         bool accumulate) {
  if (S == Scales::kE8M0)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// ---- the epilogue's stores ----------------------------------------------------------
//
// A lane has a row of the tile, so stores straight from the registers touch 32
// rows each: 6000 cycles a tile.  The warp puts 32 rows of 128 bytes (64 bf16 or
// 32 fp32 columns) into shared memory instead, 16-byte pieces swizzled by the row,
// and a bulk store takes them from there: 1300 cycles.  Where the output's rows
// do not start on 16 bytes, the warp reads the rows back and stores them itself.

constexpr int kBoxBytes = 32 * 128;

__device__ __forceinline__ void box_put(uint32_t box, int lane, int piece, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((piece ^ (lane & 7)) << 4)), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void box_store(const CUtensorMap* map, uint32_t box, int32_t col, int32_t row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(box), "r"(col), "r"(row)
               : "memory");
}

// One 128-byte piece of each of the warp's 32 rows from the sums in r (64 or 32
// columns), at (row0, col) of the output.
template <bool kF32>
__device__ __forceinline__ void store_box(const CUtensorMap* map, const PairParams& p, uint32_t box, int lane,
                                          const uint32_t* r, float alpha, int64_t row0, int64_t col) {
  constexpr int kCols = kF32 ? 32 : 64;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (kF32)
        v[e] = __float_as_uint(__uint_as_float(r[4 * j + e]) * alpha);
      else
        v[e] = pack_bf16x2(__uint_as_float(r[8 * j + 2 * e]) * alpha, __uint_as_float(r[8 * j + 2 * e + 1]) * alpha);
    }
    box_put(box, lane, j, make_uint4(v[0], v[1], v[2], v[3]));
  }
  if (p.vec) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0 && row0 < p.rows_a && col < p.rows_b)
      box_store(map, box, static_cast<int32_t>(col), static_cast<int32_t>(row0));
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  } else {
    __syncwarp();
    const int rows = static_cast<int>(min(static_cast<int64_t>(32), p.rows_a - row0));
    const int cols = static_cast<int>(min(static_cast<int64_t>(kCols), p.rows_b - col));
    for (int i = 0; i < rows; ++i) {
      const int64_t at = (row0 + i) * p.ld_out + col;
      if (kF32) {
        uint32_t v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(box + i * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4));
        if (lane < cols) reinterpret_cast<uint32_t*>(p.out)[at + lane] = v;
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = lane + 32 * h;
          uint16_t v;
          asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(box + i * 128 + (((c >> 3) ^ (i & 7)) << 4) + (c & 7) * 2));
          if (c < cols) reinterpret_cast<uint16_t*>(p.out)[at + c] = v;
        }
      }
    }
    __syncwarp();
  }
}

// ---- the kernel -----------------------------------------------------------------------

template <Scales S, bool kF32>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ CUtensorMap msa, const __grid_constant__ CUtensorMap msb,
                       const __grid_constant__ CUtensorMap mo, const PairParams p) {
  using Z = PairShape<S>;
  extern __shared__ uint8_t raw[];
  // full: the stage's loads of both CTAs (the first CTA's are waited on);
  // empty: the products that read the stage; sums: a tile's sums are complete;
  // freed: the epilogues of both CTAs have read what the next tile overwrites
  // (the first CTA's are waited on)
  __shared__ alignas(8) uint64_t bars[2 * Z::kStages + 4];
  __shared__ uint32_t tmem_addr;
  __shared__ int abort_flag;
  // for the end after a wait that ran out: loads that either CTA has issued (in the
  // first CTA), steps and tiles that the tensor cores have been given (in both)
  __shared__ int issued[2], stepped, tiled;
  // the ring starts at the same offset in both CTAs: descriptors hold for the pair
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * Z::kStages, sums = empty + 8 * Z::kStages, freed = sums + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 32) {   // kernel parameters: no earlier kernel writes them
    prefetch_tensormap(&ma);
    prefetch_tensormap(&mb);
    prefetch_tensormap(&msa);
    prefetch_tensormap(&msb);
    if (p.vec) prefetch_tensormap(&mo);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * Z::kStages + 2; ++i) mbar_init(full + 8 * i, 1);
    mbar_init(freed, 2 * kEpilogueWarps);
    mbar_init(freed + 8, 2 * kEpilogueWarps);
    fence_mbar_init();
    abort_flag = issued[0] = issued[1] = stepped = tiled = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_addr)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  cluster_sync();
  fence_after();
  grid_dependency_wait();
  grid_launch_dependents();   // after the allocation: a later kernel's cannot come first
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&tmem_addr);
  const Sync sync = {p.status, &abort_flag, p.wait_limit_ns};
  const int steps = (p.codes + kStepCodes - 1) / kStepCodes;
  const int tiles = p.tiles_a * p.tiles_b, first = blockIdx.x >> 1, stride = gridDim.x >> 1;

  if (warp == 0) {
    if (elect_one()) {
      const uint32_t full0 = at_rank(full, 0);
      const int most = static_cast<int>(rank) == p.stall_rank ? p.stall_step : INT32_MAX;
      int n = 0;   // loads so far
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const int tb = t / p.tiles_a, ta = t - tb * p.tiles_a;
        const int here = min(steps, most - n);   // (in the loop: 8192 x 14336 x 4096 176.5 us, so 174.2)
        for (int i = 0; i < here; ++i, ++n) {
          const int st = n % Z::kStages;
          if (n >= Z::kStages) ok = wait(sync, empty + 8 * st, ((n / Z::kStages) - 1) & 1);
          if (!ok) break;
          const uint32_t buf = ring + st * Z::kStage, bar = full0 + 8 * st;
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * st, 2 * Z::kStage);
          tma_load_pair(buf, &ma, bar, i * kStepBytes, ta * 256 + static_cast<int>(rank) * 128);
          tma_load_pair(buf + Z::kCodesA, &mb, bar, i * kStepBytes, tb * kN + static_cast<int>(rank) * (kN / 2));
          const uint32_t sc = buf + Z::kCodesA + Z::kCodesB;
          tma_load_pair(sc, &msa, bar, i * (Z::kScaleA / 8), ta * 2 + static_cast<int>(rank));
#pragma unroll
          for (int b = 0; b < Z::kBlocksB; ++b)
            tma_load_pair(sc + Z::kScaleA + b * Z::kScaleA, &msb, bar, i * (Z::kScaleA / 8), tb * Z::kBlocksB + b);
        }
        ok = ok && here == steps;
      }
      store_cluster(at_rank(smem_u32(&issued[rank]), 0), static_cast<uint32_t>(n));
      // every load this thread has issued has landed, or a wait has run out
      if (ok)
        for (int i = n > Z::kStages ? n - Z::kStages : 0; i < n && ok; ++i)
          ok = wait(sync, empty + 8 * (i % Z::kStages), (i / Z::kStages) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t empty1 = at_rank(empty, 1), sums1 = at_rank(sums, 1);
      int n = 0, k = 0;   // loads, tiles so far
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride, ++k) {
        // the tile before has given back the shared columns (and the one before it all)
        if (k >= 1) ok = wait(sync, freed + 8 * ((k - 1) & 1), ((k - 1) >> 1) & 1);
        fence_after();
        const uint32_t acc = tmem + ((k & 1) ? Z::kAcc1 : 0);
        for (int i = 0; i < steps && ok; ++i, ++n) {
          const int st = n % Z::kStages;
          ok = wait(sync, full + 8 * st, (n / Z::kStages) & 1);
          if (!ok) break;
          fence_after();
          const uint32_t buf = ring + st * Z::kStage;
          const uint32_t ca = tmem + Z::kScaleCol + (n & 1) * Z::kColsScale, cb = ca + Z::kColsScaleA;
          const uint64_t ds = desc_scales(buf + Z::kCodesA + Z::kCodesB);
#pragma unroll
          for (int j = 0; j < Z::kScaleTiles; ++j) {
            copy_scales_pair(ca + 4 * j, ds + 32 * j);
#pragma unroll
            for (int b = 0; b < Z::kBlocksB; ++b)
              copy_scales_pair(cb + 4 * (j * Z::kBlocksB + b), ds + (Z::kScaleA >> 4) + 32 * (b * Z::kScaleTiles + j));
          }
          const uint64_t da = desc_codes(buf), db = desc_codes(buf + Z::kCodesA);
          const int mmas = min(kMmas, (p.codes - i * kStepCodes + kMmaCodes - 1) / kMmaCodes);
#pragma unroll
          for (int j = 0; j < kMmas; ++j) {
            constexpr int kPerTile = S == Scales::kE8M0 ? 2 : 1;   // products a scale tile lasts
            if (j < mmas)
              mma_pair<S>(acc, da + 2 * j, db + 2 * j, instruction<S>(256, kN, S == Scales::kE8M0 ? 2 * (j & 1) : 0),
                          ca + 4 * (j / kPerTile), cb + 4 * (j / kPerTile) * Z::kBlocksB, i > 0 || j > 0);
          }
          commit_pair(empty + 8 * st);
          commit_pair(empty1 + 8 * st);
        }
        if (!ok) break;
        commit_pair(sums + 8 * (k & 1));
        commit_pair(sums1 + 8 * (k & 1));
      }
      for (uint32_t r = 0; r < 2; ++r) {   // (read after a barrier of the cluster, if at all)
        store_cluster(at_rank(smem_u32(&stepped), r), static_cast<uint32_t>(n));
        store_cluster(at_rank(smem_u32(&tiled), r), static_cast<uint32_t>(k));
      }
    }
  } else {
    // Two warps a quarter of the lanes take turns at the pieces of 64 columns.
    // The columns that the next tile overwrites come first (the last ones of the
    // first accumulator, the first ones of the second) and are given back once
    // they are in registers: the tensor cores wait for them.
    constexpr int kPieces = kN / 64;
    const uint32_t freed0 = at_rank(freed, 0);
    const int quarter = warp & 3, half = (warp - 2) >> 2;   // the lanes a warp may read, and which of the two it is
    Alpha alpha;
    alpha.set(p.ga, p.gb);
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t box = ring + Z::kStages * Z::kStage + (warp - 2) * kBoxBytes;
    // The round before the first (k = -1) stores nothing: while the first tile is
    // computed it brings this code into the instruction cache, which a launch
    // finds cold (1100 cycles at the end of a call that has one tile).
    for (int k = -1;; ++k) {
      const int t = first + k * stride;
      if (k >= 0 && (t >= tiles || !all_lanes(wait(sync, sums + 8 * (k & 1), (k >> 1) & 1)))) break;
      fence_after();
      const int tb = t / p.tiles_a, ta = t - tb * p.tiles_a;
      const int64_t row0 = k < 0 ? p.rows_a : static_cast<int64_t>(ta) * 256 + rank * 128 + quarter * 32;
      const int64_t col0 = static_cast<int64_t>(tb) * kN;
      const uint32_t acc = tmem + (k > 0 && (k & 1) ? Z::kAcc1 : 0) + lanes;
      const int start = (k & 1) == 0 ? Z::kAcc1 / 64 : 0;
      if (k >= 0 && half >= Z::kShared / 64) {   // none of its pieces is shared: it is done with the tile before
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(freed0 + 8 * (k & 1));
      }
#pragma unroll 1
      for (int c = half; c < (k < 0 ? half + 1 : kPieces); c += 2) {
        const int piece = (start + c) % kPieces;
        uint32_t r[64];
        load_sums32(acc + piece * 64, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        load_sums32(acc + piece * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        load_wait();
        if (k >= 0 && c < Z::kShared / 64) {
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(freed0 + 8 * (k & 1));
        }
        if (alpha.pre != 1.0f) {
#pragma unroll
          for (int e = 0; e < 64; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha.pre);
        }
#pragma unroll
        for (int h = 0; h < (kF32 ? 2 : 1); ++h) {   // an fp32 piece is two boxes
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the store before has read the box
          __syncwarp();
          store_box<kF32>(&mo, p, box, lane, &r[32 * h], alpha.last, row0, col0 + piece * 64 + 32 * h);
        }
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  // neither CTA leaves while the other may still signal its barriers or use its memory
  __syncthreads();
  if (threadIdx.x == 0 && *sync.abort) store_cluster(at_rank(smem_u32(&abort_flag), rank ^ 1), 1u);
  __syncwarp();
  cluster_sync();
  // A wait ran out, and both CTAs know: what is in flight lands before either goes on.
  // (A phase waited for here is its barrier's present one or the last: step i was
  // given to the tensor cores, and load i issued, after step i - stages was done.)
  if (*sync.abort) {
    if (threadIdx.x == 0) {
      const Drain drain;
      for (int i = max(0, stepped - Z::kStages); i < stepped; ++i)   // products, and their signals to this CTA
        drain.wait(empty + 8 * (i % Z::kStages), (i / Z::kStages) & 1);
      for (int k = max(0, tiled - 2); k < tiled; ++k) drain.wait(sums + 8 * (k & 1), (k >> 1) & 1);
      if (rank == 0) {   // loads of both CTAs; where one has not issued its half, only the other's bytes come
        const int loads = max(issued[0], issued[1]);
        for (int i = max(0, loads - Z::kStages); i < loads; ++i) {
          const uint32_t bar = full + 8 * (i % Z::kStages);
          if (i >= issued[0]) mbar_arrive_expect_tx(bar, Z::kStage);
          if (i >= issued[1]) complete_tx(bar, Z::kStage);
          drain.wait(bar, (i / Z::kStages) & 1);
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  __syncwarp();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace mm4
}  // namespace sdq
