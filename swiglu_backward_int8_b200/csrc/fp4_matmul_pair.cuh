// The large form of the product C = A B^T of two microscaled 4-bit operands
// (fp4_matmul.cuh): two multiprocessors share a tile of 256 x kN outputs
// (tcgen05.mma with cta_group::2), and a persistent grid of such pairs walks
// the tiles, a tile's sums being read out while the next one is computed.
//
// Why pairs: a CTA's half of the tile needs 128 rows of A and only its half of
// the rows of B in its own shared memory, so an instruction reads 64 bytes a
// cycle of it at the tensor cores' 4-bit rate, where a single CTA's 128 x 256
// tile would read 96 and be refilled at 100 more.
//
// Tensor memory: two accumulators of kN columns and two sets of scales.  For
// kN = 256 those do not fit, so the accumulators share columns: the second
// starts where the first still has some to go, and the epilogue of either
// reads those first and gives them back.
#pragma once

#include "fp4_matmul.cuh"

namespace sdq {
namespace mm4 {

template <Scales S, int kN>
struct PairShape {
  static constexpr int kScaleTiles = S == Scales::kE8M0 ? 2 : 4;   // a stage's scale tiles per 128 rows
  static constexpr int kBlocksB = kN / 128;
  static constexpr int kCodesA = kRows * kStepBytes;
  static constexpr int kCodesB = kN / 2 * kStepBytes;
  static constexpr int kScaleA = kScaleTiles * 512;
  static constexpr int kScaleB = kBlocksB * kScaleTiles * 512;
  static constexpr int kStage = kCodesA + kCodesB + kScaleA + kScaleB;
  static constexpr int kStages = 220 * 1024 / kStage > 8 ? 8 : 220 * 1024 / kStage;
  static constexpr int kColsScaleA = kScaleTiles * 4;
  static constexpr int kColsScale = kColsScaleA + kScaleTiles * 4 * kBlocksB;
  static constexpr int kScaleCol = 512 - 2 * kColsScale;
  static constexpr int kAcc1 = 2 * kN <= kScaleCol ? kN : (kScaleCol - kN) / 32 * 32;   // the second accumulator's first column
  static constexpr int kShared = kN - kAcc1;                                // columns both accumulators use
  static constexpr size_t kSmem = 1024 + kStages * static_cast<size_t>(kStage);
  static_assert(kStage % 1024 == 0, "the swizzled boxes start on 1024 bytes");
  static_assert(kAcc1 >= 0 && kAcc1 % 32 == 0 && kShared % 32 == 0, "whole 32-column chunks");
};

struct PairParams {
  const float* ga;
  const float* gb;
  uint8_t* out;
  int64_t ld_out;
  int64_t rows_a, rows_b;
  int32_t codes;
  int32_t tiles_a, tiles_b;
  int32_t out_f32;
  int32_t vec;             // bytes a store may have: 32, 16 or 0 (an element)
  int* status;
  uint64_t wait_limit_ns;
};

// ---- pairs ------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
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

// As instruction(), for 256 rows.
template <Scales S, int kN>
__device__ __forceinline__ uint32_t instruction_pair(uint32_t scale_byte) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kN / 8) << 17) | (S == Scales::kE8M0 ? 1u << 23 : 0u) |
         (2u << 27) | (scale_byte << 4) | (scale_byte << 29);
}

// ---- the epilogue's stores ----------------------------------------------------------

__device__ __forceinline__ void store_bytes32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 columns of a row; n of them exist.  A lane has a row, so a store of 32
// bytes is the widest that fills whole sectors.
__device__ __forceinline__ void store_columns(uint8_t* row, int64_t col, int n, const uint32_t (&r)[32], float alpha,
                                              int f32, int vec) {
  if (f32) {
    float* o = reinterpret_cast<float*>(row) + col;
    if (vec && n >= 32) {
      uint32_t v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
      if (vec == 32) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) store_bytes32(o + e, v + e);
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4*>(o + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (e < n) o[e] = __uint_as_float(r[e]) * alpha;
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(row) + col;
    uint32_t v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      v[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * alpha, __uint_as_float(r[2 * e + 1]) * alpha);
    if (vec && n >= 32) {
      if (vec == 32) {
        store_bytes32(o, v);
        store_bytes32(o + 16, v + 8);
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(o + 2 * e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (e < n) o[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// ---- the kernel -----------------------------------------------------------------------

template <Scales S, int kN>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ CUtensorMap msa, const __grid_constant__ CUtensorMap msb,
                       const PairParams p) {
  using Z = PairShape<S, kN>;
  extern __shared__ uint8_t raw[];
  // full: the stage's loads of both CTAs (the first CTA's are waited on);
  // empty: the products that read the stage; sums: a tile's sums are complete;
  // freed: the epilogues of both CTAs have read what the next tile overwrites
  // (the first CTA's are waited on)
  __shared__ alignas(8) uint64_t bars[2 * Z::kStages + 4];
  __shared__ uint32_t tmem_addr;
  __shared__ int abort_flag;
  // the ring starts at the same offset in both CTAs: descriptors hold for the pair
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8 * Z::kStages, sums = empty + 8 * Z::kStages, freed = sums + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * Z::kStages + 2; ++i) mbar_init(full + 8 * i, 1);
    mbar_init(freed, 8);
    mbar_init(freed + 8, 8);
    fence_mbar_init();
    abort_flag = 0;
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
      int n = 0;   // loads so far
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const int tb = t / p.tiles_a, ta = t - tb * p.tiles_a;
        for (int i = 0; i < steps; ++i, ++n) {
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
      }
      // every load this thread has issued has landed, or its wait has run out
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
        if (Z::kShared > 0) {   // the tile before has given back the shared columns
          if (k >= 1) ok = wait(sync, freed + 8 * ((k - 1) & 1), ((k - 1) >> 1) & 1);
        } else {                // the tile before that is read out
          if (k >= 2) ok = wait(sync, freed + 8 * (k & 1), ((k - 2) >> 1) & 1);
        }
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
              mma_pair<S>(acc, da + 2 * j, db + 2 * j, instruction_pair<S, kN>(S == Scales::kE8M0 ? 2 * (j & 1) : 0),
                          ca + 4 * (j / kPerTile), cb + 4 * (j / kPerTile) * Z::kBlocksB, i > 0 || j > 0);
          }
          commit_pair(empty + 8 * st);
          commit_pair(empty1 + 8 * st);
        }
        if (ok) {
          commit_pair(sums + 8 * (k & 1));
          commit_pair(sums1 + 8 * (k & 1));
        }
      }
    }
  } else {
    const uint32_t freed0 = at_rank(freed, 0);
    const int quarter = warp & 3;   // the lanes a warp may read
    const float alpha = (p.ga ? *p.ga : 1.0f) * (p.gb ? *p.gb : 1.0f);
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int k = 0;
    for (int t = first; t < tiles; t += stride, ++k) {
      if (!wait(sync, sums + 8 * (k & 1), (k >> 1) & 1)) break;
      fence_after();
      const int tb = t / p.tiles_a, ta = t - tb * p.tiles_a;
      const int64_t row = static_cast<int64_t>(ta) * 256 + rank * 128 + quarter * 32 + lane;
      const int64_t col0 = static_cast<int64_t>(tb) * kN;
      uint8_t* o = p.out + row * p.ld_out * (p.out_f32 ? 4 : 2);
      const uint32_t acc = tmem + ((k & 1) ? Z::kAcc1 : 0) + lanes;
      constexpr int kChunks = kN / 32;
      // the columns that the next tile overwrites come first: the last ones of
      // the first accumulator, the first ones of the second
      const int start = Z::kShared > 0 && (k & 1) == 0 ? Z::kAcc1 / 32 : 0;
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int cc = start + c < kChunks ? start + c : start + c - kChunks;
        uint32_t r[32];
        load_sums32(acc + cc * 32, r);
        load_wait();
        if (Z::kShared > 0 ? c == Z::kShared / 32 - 1 : c == kChunks - 1) {
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(freed0 + 8 * (k & 1));
        }
        const int64_t n = p.rows_b - col0 - cc * 32;
        if (row < p.rows_a && n > 0)
          store_columns(o, col0 + cc * 32, static_cast<int>(n < 32 ? n : 32), r, alpha, p.out_f32, p.vec);
      }
    }
  }
  // neither CTA leaves while the other may still signal its barriers or use its memory
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {   // a wait ran out: give what is in flight the same time to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < p.wait_limit_ns) __nanosleep(1000);
  }
  __syncthreads();
  cluster_sync();
  __syncwarp();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace mm4
}  // namespace sdq
