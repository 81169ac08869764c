// Products on the tensor cores, with the element-wise part of an operator as
// their epilogue.
//
// One CTA per SM takes tiles of 128 x tn.  A warp's lane fills four stages of
// shared memory by TMA, 64 places of the sum at a time; a lane of another warp
// issues the tcgen05 products of the stages that have arrived, with the
// accumulators in tensor memory; four more warps take a finished tile from
// there (mm_epilogue.cuh) while the next one is being summed into the other half
// of the 512 columns.
//
// Where a product has fewer tiles than there are SMs, each tile's sum is cut into
// splits that different CTAs take; they leave fp32 sums in the workspace, and a
// second kernel adds these in order and runs the epilogue.
#include "mm_epilogue.cuh"
#include "mm_tcgen05.cuh"

namespace vcoll {

namespace {

// Tiles in groups of 16 rows of tiles: the tiles that are in flight together
// share their operands through the L2.
constexpr int kGroup = 16;
__device__ __forceinline__ void tile_at(const MmParams& p, int64_t tile, int64_t& m, int64_t& n) {
  const int64_t per = kGroup * p.tiles_n;
  const int64_t g = tile / per, in = tile % per;
  const int64_t rows = p.tiles_m - g * kGroup < kGroup ? p.tiles_m - g * kGroup : kGroup;
  m = g * kGroup + in % rows;
  n = in / rows;
}

}  // namespace

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kMmThreads, 1) vc_mm(const __grid_constant__ MmParams p) {
  pdl_enter();
  extern __shared__ unsigned char raw[];
  __shared__ volatile int gave_up;
  __shared__ uint32_t tmem_at;
  const uint32_t base = (mm_smem(raw) + 1023) & ~1023u;  // of 128-byte swizzle atoms
  const uint32_t stage0 = base, blocks = base + kMmStages * (kMmStageA + kMmStageB);
  const uint32_t bars = blocks + kMmEpilogueBytes;
  const uint32_t full = bars, empty = bars + 8 * kMmStages, acc_full = empty + 8 * kMmStages,
                 acc_empty = acc_full + 16, drained = acc_empty + 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const MmAbort guard = {&gave_up, p.error_word};
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMmStages; ++s) {
      mm_bar_init(full + 8 * s, 1);
      mm_bar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mm_bar_init(acc_full + 8 * s, 1);
      mm_bar_init(acc_empty + 8 * s, kMmEpilogueWarps);
    }
    mm_bar_init(drained, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmEpilogueWarps + 1) mm_tmem_alloc<2 * kMmTileN>(mm_smem(&tmem_at));
  mm_fence_before();
  __syncthreads();
  mm_fence_after();
  const uint32_t tmem = tmem_at;

  const int64_t units = p.tiles_m * p.tiles_n * p.splits;
  const int64_t depth = (p.K + kMmDepth - 1) / kMmDepth;  // steps of a sum
  const int64_t steps = mm_pairs(p.parts) * depth;

  if (warp == kMmEpilogueWarps) {
    if (lane == 0) {
      int64_t issued = 0;
      const int64_t second = p.K1 / kMmDepth;  // the first step that takes map_b[1]
      for (int64_t u = blockIdx.x; u < units && !gave_up; u += gridDim.x) {
        int64_t tm, tn;
        tile_at(p, u / p.splits, tm, tn);
        const int64_t s = u % p.splits;
        const int64_t begin = steps * s / p.splits, end = steps * (s + 1) / p.splits;
        int64_t q = begin / (depth ? depth : 1), k = begin - q * depth;
        for (int64_t i = begin; i < end; ++i, ++issued) {
          const int st = issued % kMmStages;
          if (issued >= kMmStages && !mm_bar_wait(empty + 8 * st, (issued / kMmStages - 1) & 1, guard)) break;
          const uint32_t a = stage0 + st * (kMmStageA + kMmStageB), b = a + kMmStageA, bar = full + 8 * st;
          mm_bar_expect(bar, kMmStageA + p.tn * kMmDepth * 2);
          const int pa = mm_pair_a(mm_pairs(p.parts), q), pb = mm_pair_b(mm_pairs(p.parts), q);
          const int kk = (int)(k * kMmDepth);
          if (A_MN) {
            for (int c = 0; c < kMmTileM / 64; ++c)
              mm_load_box(a + c * 8192, &p.map_a, (int)(tm * kMmTileM) + 64 * c, kk, pa, bar);
          } else {
            mm_load_box(a, &p.map_a, kk, (int)(tm * kMmTileM), pa, bar);
          }
          if (EPI == MM_GATED) {
            for (int h = 0; h < 2; ++h)
              mm_load_box(b + h * (p.tn / 2) * kMmDepth * 2, &p.map_b[h], kk, (int)(tn * (p.tn / 2)), pb, bar);
          } else if (B_MN) {
            const CUtensorMap* map = &p.map_b[k >= second];
            const int kb = kk - (k >= second ? (int)p.K1 : 0);
            for (int c = 0; c < p.tn / 64; ++c)
              mm_load_box(b + c * 8192, map, (int)(tn * p.tn) + 64 * c, kb, pb, bar);
          } else {
            mm_load_box(b, &p.map_b[0], kk, (int)(tn * p.tn), pb, bar);
          }
          if (++k == depth) {
            k = 0;
            ++q;
          }
        }
      }
      if (gave_up)  // copies cannot be called back: their memory has to stay until they have landed
        for (int64_t i = issued < kMmStages ? 0 : issued - kMmStages; i < issued; ++i)
          mm_bar_wait(full + 8 * (i % kMmStages), (i / kMmStages) & 1, guard, kMmDrainNs);
    }
  } else if (warp == kMmEpilogueWarps + 1) {
    if (lane == 0) {
      const uint32_t idesc = mm_idesc(A_MN, B_MN, kMmTileM, p.tn);
      int64_t done = 0, it = 0;
      for (int64_t u = blockIdx.x; u < units && !gave_up; u += gridDim.x, ++it) {
        const int64_t s = u % p.splits;
        const int64_t count = steps * (s + 1) / p.splits - steps * s / p.splits;
        const int acc = it & 1;
        if (!mm_bar_wait(acc_empty + 8 * acc, ((it >> 1) & 1) ^ 1, guard)) break;
        mm_fence_after();
        const uint32_t d = tmem + acc * kMmTileN;
        bool ok = true;
        for (int64_t i = 0; i < count && ok; ++i, ++done) {
          const int st = done % kMmStages;
          ok = mm_bar_wait(full + 8 * st, (done / kMmStages) & 1, guard);
          if (!ok) break;
          mm_fence_after();
          const uint32_t a = stage0 + st * (kMmStageA + kMmStageB);
          const uint64_t da = mm_desc(a, A_MN), db = mm_desc(a + kMmStageA, B_MN);
#pragma unroll
          for (int j = 0; j < kMmDepth / 16; ++j)
            mm_mma(d, da + j * mm_desc_step(A_MN), db + j * mm_desc_step(B_MN), idesc, i > 0 || j > 0);
          mm_commit(empty + 8 * st);
        }
        if (!ok) break;
        mm_commit(acc_full + 8 * acc);
      }
      if (gave_up) {
        mm_commit(drained);
        mm_bar_wait(drained, 0, guard, kMmDrainNs);
      }
    }
  } else {
    float* stage = reinterpret_cast<float*>(raw + (blocks - mm_smem(raw))) + warp * 2 * kMmBlockWords;
    int64_t it = 0;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++it) {
      const int acc = it & 1;
      if (!__all_sync(~0u, mm_bar_wait(acc_full + 8 * acc, (it >> 1) & 1, guard))) break;
      mm_fence_after();
      int64_t tm, tn;
      tile_at(p, u / p.splits, tm, tn);
      const uint32_t d = tmem + ((uint32_t)(warp * 32) << 16) + acc * kMmTileN;
      auto src = [&](int c, float (&v)[32]) {
        mm_tmem_load(d + c, v);
        if (!steps) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        }
      };
      const int64_t row0 = tm * kMmTileM + warp * 32;
      if (p.splits == 1) {
        mm_epilogue<EPI>(p, row0, tn, lane, stage, src);
      } else {
        const int64_t rows = p.M < kMmTileM ? p.M : kMmTileM;
        float4* to = reinterpret_cast<float4*>(p.partial + (u * rows + warp * 32 + lane) * p.tn);
        for (int c = 0; c < p.tn; c += 32) {
          float v[32];
          src(c, v);
          if (row0 + lane < p.M) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              to[c / 4 + j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
      }
      mm_fence_before();
      __syncwarp();
      if (lane == 0) mm_bar_arrive(acc_empty + 8 * acc);
    }
  }
  __syncwarp();
  mm_fence_before();
  __syncthreads();
  if (warp == kMmEpilogueWarps + 1) mm_tmem_free<2 * kMmTileN>(tmem);
}

// The epilogue of a tile whose sum was cut: the splits' sums added in order.
template <int EPI>
__global__ void __launch_bounds__(kMmEpilogueWarps * 32) vc_mm_join_splits(const __grid_constant__ MmParams p) {
  pdl_enter();
  __shared__ float blocks[kMmEpilogueWarps * 2 * kMmBlockWords];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t tile = blockIdx.x;
  int64_t tm, tn;
  tile_at(p, tile, tm, tn);
  const int64_t row0 = tm * kMmTileM + warp * 32;
  if (row0 >= p.M) return;
  const int64_t rows = p.M < kMmTileM ? p.M : kMmTileM;
  const float* from = p.partial + (tile * p.splits * rows + warp * 32 + lane) * p.tn;
  mm_epilogue<EPI>(p, row0, tn, lane, blocks + warp * 2 * kMmBlockWords, [&](int c, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    if (row0 + lane >= p.M) return;
    for (int s = 0; s < p.splits; ++s) {
      const float4* q = reinterpret_cast<const float4*>(from + s * rows * p.tn + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 x = q[j];
        v[4 * j] += x.x;
        v[4 * j + 1] += x.y;
        v[4 * j + 2] += x.z;
        v[4 * j + 3] += x.w;
      }
    }
  });
}

const void* mm_kernel(MmEpilogue epilogue, bool a_mn) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm<MM_LSE, false, false>;
    case MM_ERROR:
      return (const void*)vc_mm<MM_ERROR, false, false>;
    case MM_GATED:
      return (const void*)vc_mm<MM_GATED, false, false>;
    default:
      return a_mn ? (const void*)vc_mm<MM_OUT, true, true> : (const void*)vc_mm<MM_OUT, false, true>;
  }
}

const void* mm_join_splits_kernel(MmEpilogue epilogue) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm_join_splits<MM_LSE>;
    case MM_ERROR:
      return (const void*)vc_mm_join_splits<MM_ERROR>;
    case MM_GATED:
      return (const void*)vc_mm_join_splits<MM_GATED>;
    default:
      return (const void*)vc_mm_join_splits<MM_OUT>;
  }
}

}  // namespace vcoll
