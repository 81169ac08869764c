// Products on the tensor cores, with the element-wise part of an operator as
// their epilogue.
//
// One CTA per SM, or a pair of CTAs on two SMs, takes tiles of 128 or 256 rows
// and up to 256 columns.  A warp's lane fills stages of shared memory by TMA, 64
// places of the sum at a time; a lane of another warp (of a pair: of its first
// CTA) issues the tcgen05 products of the stages that have arrived, with the
// accumulators in tensor memory; four more warps take a finished tile from there
// (mm_epilogue.cuh) while the next one is being summed into the other half of
// the 512 columns.  Each CTA of a pair holds half of the columns' operand, which
// the products of both read: that takes a third less from L2 and shared memory.
//
// Where a product has fewer tiles than there are SMs, each tile's sum is cut into
// splits that different CTAs take; they leave fp32 sums in the workspace, and a
// second kernel adds these in order and runs the epilogue.
#include "mm_epilogue.cuh"
#include "mm_tcgen05.cuh"

namespace vcoll {

namespace {

// Tiles in groups of 2048 rows: the tiles that are in flight together share their
// operands through the L2.
__device__ __forceinline__ void tile_at(const MmParams& p, int tile_rows, int64_t tile, int64_t& m, int64_t& n) {
  const int64_t group = 2048 / tile_rows, per = group * p.tiles_n;
  const int64_t g = tile / per, in = tile % per;
  const int64_t rows = p.tiles_m - g * group < group ? p.tiles_m - g * group : group;
  m = g * group + in % rows;
  n = in / rows;
}

}  // namespace

template <int EPI, bool A_MN, bool B_MN, int CTAS>
__global__ void __launch_bounds__(kMmThreads, 1) vc_mm(const __grid_constant__ MmParams p) {
  pdl_enter();
  extern __shared__ unsigned char raw[];
  __shared__ volatile int gave_up;
  __shared__ uint32_t tmem_at;
  constexpr int TILE_ROWS = kMmRows * CTAS;
  const uint32_t stage0 = (mm_smem(raw) + 1023) & ~1023u;  // of 128-byte swizzle atoms
  const uint32_t blocks = stage0 + kMmStageRoom, bars = blocks + kMmEpilogueBytes;
  const uint32_t full = bars, empty = bars + 8 * kMmMaxStages, acc_full = empty + 8 * kMmMaxStages,
                 acc_empty = acc_full + 16, drained = acc_empty + 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CTAS == 1 ? 0 : mm_rank();
  const MmAbort guard = {&gave_up, p.error_word};
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMmMaxStages; ++s) {
      mm_bar_init(full + 8 * s, 1);
      mm_bar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mm_bar_init(acc_full + 8 * s, 1);
      mm_bar_init(acc_empty + 8 * s, kMmEpilogueWarps * CTAS);
    }
    mm_bar_init(drained, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmEpilogueWarps + 1) mm_tmem_alloc<CTAS>(mm_smem(&tmem_at));
  mm_fence_before();
  __syncthreads();
  if (CTAS > 1) mm_cluster_sync();
  mm_fence_after();
  const uint32_t tmem = tmem_at;

  const int64_t units = p.tiles_m * p.tiles_n * p.splits;
  const int64_t first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;
  const int64_t depth = (p.K + kMmDepth - 1) / kMmDepth;  // steps of a sum
  const int pairs = mm_pairs(p.parts);
  const int64_t steps = pairs * depth;
  const int stages = p.stages;
  const int stage_a = p.a_rows * kMmDepth * 2;

  if (warp == kMmEpilogueWarps) {
    if (lane == 0) {
      const int64_t second = p.K1 / kMmDepth;  // the first step that takes map_b[1]
      const int cols = p.tn / CTAS;            // of b that this CTA holds
      const uint32_t bytes = (uint32_t)CTAS * (stage_a + cols * kMmDepth * 2);
      int64_t issued = 0;
      int st = 0, round = 0;
      for (int64_t u = first; u < units && !gave_up; u += stride) {
        int64_t tm, tn;
        tile_at(p, TILE_ROWS, u / p.splits, tm, tn);
        const int64_t s = u % p.splits;
        const int64_t begin = steps * s / p.splits, end = steps * (s + 1) / p.splits;
        int q = depth ? (int)(begin / depth) : 0;
        int64_t k = begin - q * depth;
        const int row = (int)(tm * TILE_ROWS) + (int)rank * kMmRows;
        const int col = EPI == MM_GATED ? (int)(tn * (p.tn / 2)) : (int)(tn * p.tn) + (int)rank * cols;
        for (int64_t i = begin; i < end; ++i, ++issued) {
          if (round && !mm_bar_wait(empty + 8 * st, (round - 1) & 1, guard)) break;
          const uint32_t a = stage0 + st * p.stage_bytes, b = a + stage_a;
          uint32_t bar = full + 8 * st;
          if (rank == 0) mm_bar_expect(bar, bytes);
          if (CTAS > 1) bar = mm_of_first(bar);
          const int pa = mm_pair_a(pairs, q), pb = mm_pair_b(pairs, q);
          const int kk = (int)(k * kMmDepth);
          if (A_MN) {
            for (int c = 0; c < kMmRows / 64; ++c)
              mm_load_box<CTAS>(a + c * 8192, &p.map_a, row + 64 * c, kk, pa, bar);
          } else {
            mm_load_box<CTAS>(a, &p.map_a, kk, row, pa, bar);
          }
          if (EPI == MM_GATED && CTAS == 2) {
            mm_load_box<CTAS>(b, &p.map_b[rank], kk, col, pb, bar);
          } else if (EPI == MM_GATED) {
            for (int h = 0; h < 2; ++h)
              mm_load_box<CTAS>(b + h * (p.tn / 2) * kMmDepth * 2, &p.map_b[h], kk, col, pb, bar);
          } else if (B_MN) {
            const CUtensorMap* map = &p.map_b[k >= second];
            const int kb = kk - (k >= second ? (int)p.K1 : 0);
            for (int c = 0; c < cols / 64; ++c)
              mm_load_box<CTAS>(b + c * 8192, map, col + 64 * c, kb, pb, bar);
          } else {
            mm_load_box<CTAS>(b, &p.map_b[0], kk, col, pb, bar);
          }
          if (++k == depth) {
            k = 0;
            ++q;
          }
          if (++st == stages) {
            st = 0;
            ++round;
          }
        }
      }
      if (gave_up && rank == 0)  // copies cannot be called back: their memory has to stay until they have landed
        for (int64_t i = issued < stages ? 0 : issued - stages; i < issued; ++i)
          mm_bar_wait(full + 8 * (i % stages), (i / stages) & 1, guard, kMmDrainNs);
    }
  } else if (warp == kMmEpilogueWarps + 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = mm_idesc(A_MN, B_MN, TILE_ROWS, p.tn);
      int64_t it = 0;
      int st = 0, round = 0;
      for (int64_t u = first; u < units && !gave_up; u += stride, ++it) {
        const int64_t s = u % p.splits;
        const int64_t count = steps * (s + 1) / p.splits - steps * s / p.splits;
        const int acc = it & 1;
        if (!mm_bar_wait(acc_empty + 8 * acc, ((it >> 1) & 1) ^ 1, guard)) break;
        mm_fence_after();
        const uint32_t d = tmem + acc * kMmTileN;
        bool ok = true;
        for (int64_t i = 0; i < count; ++i) {
          ok = mm_bar_wait(full + 8 * st, round & 1, guard);
          if (!ok) break;
          mm_fence_after();
          const uint32_t a = stage0 + st * p.stage_bytes;
          const uint64_t da = mm_desc(a, A_MN), db = mm_desc(a + stage_a, B_MN);
#pragma unroll
          for (int j = 0; j < kMmDepth / 16; ++j)
            mm_mma<CTAS>(d, da + j * mm_desc_step(A_MN), db + j * mm_desc_step(B_MN), idesc, i > 0 || j > 0);
          mm_commit<CTAS>(empty + 8 * st);
          if (++st == stages) {
            st = 0;
            ++round;
          }
        }
        if (!ok) break;
        mm_commit<CTAS>(acc_full + 8 * acc);
      }
      if (gave_up) {
        mm_commit<CTAS>(drained);
        mm_bar_wait(drained, 0, guard, kMmDrainNs);
      }
    }
  } else {
    uint32_t* block = reinterpret_cast<uint32_t*>(raw + (blocks - mm_smem(raw))) + warp * kMmBlockWords;
    int64_t it = 0;
    for (int64_t u = first; u < units; u += stride, ++it) {
      const int acc = it & 1;
      if (!__all_sync(~0u, mm_bar_wait(acc_full + 8 * acc, (it >> 1) & 1, guard))) break;
      mm_fence_after();
      int64_t tm, tn;
      tile_at(p, TILE_ROWS, u / p.splits, tm, tn);
      const uint32_t d = tmem + ((uint32_t)(warp * 32) << 16) + acc * kMmTileN;
      auto src = [&](int c0, int c1, float (&x)[32], float (&y)[32]) {
        uint32_t r0[32], r1[32];
        mm_tmem_load(d + c0, r0);
        mm_tmem_load(d + c1, r1);
        mm_tmem_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          x[j] = steps ? __uint_as_float(r0[j]) : 0.0f;  // nothing was summed
          y[j] = steps ? __uint_as_float(r1[j]) : 0.0f;
        }
      };
      const int in_tile = (int)rank * kMmRows + warp * 32;
      const int64_t row0 = tm * TILE_ROWS + in_tile;
      if (p.splits == 1) {
        mm_epilogue<EPI>(p, row0, tn, lane, block, src);
      } else {
        const int64_t rows = p.M < TILE_ROWS ? p.M : TILE_ROWS;
        float4* to = reinterpret_cast<float4*>(p.partial + (u * rows + in_tile + lane) * p.tn);
        for (int c = 0; c < p.tn; c += 64) {
          float x[32], y[32];
          src(c, c + 32, x, y);
          if (row0 + lane < p.M) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              to[c / 4 + j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
              to[c / 4 + 8 + j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
            }
          }
        }
      }
      mm_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 1)
          mm_bar_arrive(acc_empty + 8 * acc);
        else
          mm_bar_arrive_at(mm_of_first(acc_empty + 8 * acc));
      }
    }
  }
  __syncwarp();
  mm_fence_before();
  __syncthreads();
  if (CTAS > 1) mm_cluster_sync();  // the other CTA's copies and products reach into this one's memory
  if (warp == kMmEpilogueWarps + 1) mm_tmem_free<CTAS>(tmem);
}

// The epilogue of tiles whose sums were cut: the splits' sums added in order, a
// warp for 32 columns of a row (MM_LSE: for a tile's).
template <int EPI>
__global__ void __launch_bounds__(256) vc_mm_join_splits(const __grid_constant__ MmParams p) {
  pdl_enter();
  const int lane = threadIdx.x % 32;
  const int tile_rows = p.tile_rows;
  const int64_t rows = p.M < tile_rows ? p.M : tile_rows;
  const int width = EPI == MM_GATED ? p.tn / 2 : p.tn, chunks = EPI == MM_LSE ? 1 : width / 32;
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  const int chunk = (int)(w % chunks);
  const int64_t r = w / chunks % rows, tile = w / chunks / rows;
  if (tile >= p.tiles_m * p.tiles_n) return;
  int64_t tm, tn;
  tile_at(p, tile_rows, tile, tm, tn);
  const int64_t row = tm * tile_rows + r;
  if (row >= p.M) return;
  const float* from = p.partial + (tile * p.splits * rows + r) * p.tn;
  auto sum = [&](int c) {
    float x = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) x += from[s * rows * p.tn + c];
    return x;
  };
  const int c = chunk * 32 + lane;
  const int64_t col = tn * width + c;
  if constexpr (EPI == MM_OUT) {
    const MmOutRow to = mm_out_row(p, row);
    if (col >= p.N || to.row >= (p.M1 ? p.M2 : p.M)) return;
    float x = sum(c);
    if (p.accum_in) x += p.accum_in[row * p.accum_ld + col];
    if (p.accum_out) {
      p.accum_out[row * p.accum_ld + col] = x;
      return;
    }
    if (p.scale) x *= *p.scale;
    if (p.base) x += mm_load(p.base, p.out_f32, to.row * p.base_ld + col);
    mm_store(to.out, p.out_f32, to.row * to.ld + col, x);
  } else if constexpr (EPI == MM_LSE) {
    const int64_t t = mm_token(p.targets, p.idx64, row);
    const int64_t hit = t >= 0 && t < p.V ? t - p.token0 : -1;
    float v[kMmTileN / 32], top = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMmTileN / 32; ++i) {
      const int64_t at = tn * p.tn + i * 32 + lane;
      const bool in = i * 32 < p.tn && at < p.N;
      v[i] = in ? sum(i * 32 + lane) : -INFINITY;
      if (in && at == hit) p.picked[row] = v[i];
      top = fmaxf(top, v[i]);
    }
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    top *= kMmLog2e;
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < kMmTileN / 32; ++i) s += mm_exp2(fmaf(v[i], kMmLog2e, -ref));
    for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
    if (lane == 0) p.part[tn * p.M + row] = make_float2(top, s);
  } else if constexpr (EPI == MM_ERROR) {
    if (col >= p.N) return;
    const int64_t t = mm_token(p.targets, p.idx64, row);
    float x = 0.0f;
    if (t >= 0 && t < p.V) {
      x = mm_exp(sum(c) - p.lse[row]);
      if (t - p.token0 == col) x -= 1.0f;
      x *= p.dloss[row * p.dloss_step] / *p.scale;
    }
    uint16_t* to = static_cast<uint16_t*>(p.error) + row * p.error_ld + col;
    for (int k = 0; k < p.parts; ++k) {
      to[k * p.error_plane] = mm_narrow(x);
      x -= Elem<__nv_bfloat16>::widen1(mm_narrow(x));
    }
  } else {
    if (col >= p.N) return;
    const float g = sum(c), u = sum(width + c);
    float s, ds;
    mm_act(p.act, g, s, ds);
    if (p.gate) mm_store(p.gate, p.out_f32, row * p.gate_ld + col, g);
    if (p.up) mm_store(p.up, p.out_f32, row * p.up_ld + col, u);
    mm_store(p.out, p.out_f32, row * p.out_ld + col, g * (s * u));
  }
}

template <int CTAS>
static const void* kernel_of(MmEpilogue epilogue, bool a_mn) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm<MM_LSE, false, false, CTAS>;
    case MM_ERROR:
      return (const void*)vc_mm<MM_ERROR, false, false, CTAS>;
    case MM_GATED:
      return (const void*)vc_mm<MM_GATED, false, false, CTAS>;
    default:
      return a_mn ? (const void*)vc_mm<MM_OUT, true, true, CTAS> : (const void*)vc_mm<MM_OUT, false, true, CTAS>;
  }
}

const void* mm_kernel(MmEpilogue epilogue, bool a_mn, int ctas) {
  return ctas == 2 ? kernel_of<2>(epilogue, a_mn) : kernel_of<1>(epilogue, a_mn);
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
