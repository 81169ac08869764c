// Products on the tensor cores, with the element-wise part of an operator as
// their epilogue.
//
// One CTA per SM, or a pair of CTAs on two SMs, takes tiles of 128 or 256 rows
// and up to 256 columns.  A warp's lane fills stages of shared memory by TMA, 64
// places of the sum at a time; a lane of another warp (of a pair: of its first
// CTA) issues the tcgen05 products of the stages that have arrived, with the
// accumulators in tensor memory; eight more warps take a finished tile from there
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

// Tiles in groups of rows, column after column: the tiles that are in flight together
// share their operands through the L2.
__device__ __forceinline__ void tile_at(const MmParams& p, uint32_t tile, uint32_t& m, uint32_t& n) {
  const uint32_t group = p.group, per = group * p.tiles_n;
  const uint32_t g = tile / per, in = tile - g * per;
  const uint32_t rows = p.tiles_m - g * group < group ? p.tiles_m - g * group : group;
  n = in / rows;
  m = g * group + in - n * rows;
}

// What a CTA (or pair) does n-th: a unit of one of the launch's products.
struct Unit {
  bool second;
  uint32_t at;
};
template <bool TWO>
__device__ __forceinline__ bool unit_at(const MmLaunch& all, uint32_t me, uint32_t of, uint32_t n, Unit& u) {
  const uint32_t units = all.p[0].units;
  if (!TWO) {
    u = {false, n * of + me};
    return u.at < units;
  }
  const uint32_t more = units % of, mine = units / of + (me < more);
  if (n < mine) {
    u = {false, n * of + me};
    return true;
  }
  n -= mine;
  u.second = true;
  if (me >= more && n < all.ahead) {
    u.at = n * (of - more) + me - more;
  } else {
    if (me >= more) n -= all.ahead;
    u.at = all.ahead * (of - more) + n * of + me;
  }
  return u.at < all.p[1].units;
}

// A unit's tile, and its steps: of every pair of parts' `depth` steps a split takes
// every splits-th, so that the splits of a tile, which run side by side, read
// memory that lies side by side.
__device__ __forceinline__ uint32_t steps_of(const MmParams& p, uint32_t unit, uint32_t& tile, uint32_t& split) {
  const uint32_t steps = mm_pairs(p.parts) * p.depth;
  tile = unit;
  split = 0;
  if (p.splits == 1) return steps;
  tile = unit / p.splits;
  split = unit - tile * p.splits;
  return (steps - split + p.splits - 1) / p.splits;
}

// Steps of a unit's first chunk: the small ones of the parts' products together.
__device__ __forceinline__ uint32_t first_chunk(const MmParams& p, uint32_t split) {
  if (p.parts < 3) return p.chunk;
  const uint32_t small = ((mm_pairs(p.parts) - 1) * p.depth - split + p.splits - 1) / p.splits;
  return small < kMmChunkMost ? small : kMmChunkMost;
}

// Where a CTA's parts lie in shared memory, and its place in a pair.
struct Place {
  uint32_t stage0, full, empty, acc_full, acc_empty, drained;
  uint32_t rank, tmem;
  int stages, stage_bytes;
  MmAbort guard;
};
struct Ring {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
};

// A unit's copies into the ring, by a whole warp of which one lane issues them; the
// number of stages that were filled.  A step lasts 512
// cycles at 256 columns and 256 at 128: what does not change is outside the loop.
template <int EPI, int CTAS, bool A_MN>
__device__ __forceinline__ uint32_t load_unit(const MmParams& p, uint32_t unit, const Place& at, Ring& ring) {
  constexpr int TILE_ROWS = kMmRows * CTAS;
  constexpr bool B_MN = EPI == MM_OUT;
  const int cols = p.tn / CTAS;  // of b that this CTA holds
  const int stage_a = p.a_rows * kMmDepth * 2, half_b = p.tn / 2 * kMmDepth * 2;
  const uint32_t bytes = (uint32_t)CTAS * (stage_a + cols * kMmDepth * 2);
  const int pairs = mm_pairs(p.parts);
  const uint32_t depth = p.depth, stride = p.splits;
  const uint32_t second = B_MN ? (uint32_t)(p.K1 / kMmDepth) : 0;  // the first step that takes map_b[1]
  uint32_t tile, tm, tn, k, done = 0;
  steps_of(p, unit, tile, k);
  tile_at(p, tile, tm, tn);
  const int row = (int)(tm * TILE_ROWS + at.rank * kMmRows);
  const int col = EPI == MM_GATED ? (int)(tn * (p.tn / 2)) : (int)(tn * p.tn + at.rank * cols);
  const CUtensorMap *map_a = &p.map_a, *map_b = EPI == MM_GATED && CTAS == 2 && at.rank ? &p.map_b[1] : &p.map_b[0];
  const uint32_t signal = CTAS > 1 ? mm_of_first(at.full) : at.full;
  for (int q = 0; q < pairs; ++q, k -= depth) {
    const int pa = mm_pair_a(pairs, q), pb = mm_pair_b(pairs, q);
    for (; k < depth; k += stride, ++done) {
      // an empty stage's barrier was never used: the phase before its first is over
      if (!mm_warp_wait(at.empty + 8 * ring.stage, (ring.round & 1) ^ 1, at.guard)) return done;
      const uint32_t a = at.stage0 + ring.stage * at.stage_bytes, b = a + stage_a, bar = signal + 8 * ring.stage;
      const uint32_t mine = at.full + 8 * ring.stage;
      ring.next(at.stages);
      const int kk = (int)(k * kMmDepth);
      if (!mm_elect()) continue;
      if (CTAS == 1 || at.rank == 0) mm_bar_expect(mine, bytes);
      if (A_MN) {
#pragma unroll
        for (int c = 0; c < kMmRows / 64; ++c) mm_load_box<CTAS>(a + c * 8192, map_a, row + 64 * c, kk, pa, bar);
      } else {
        mm_load_box<CTAS>(a, map_a, kk, row, pa, bar);
      }
      if (EPI == MM_GATED && CTAS == 1) {
        mm_load_box<CTAS>(b, &p.map_b[0], kk, col, pb, bar);
        mm_load_box<CTAS>(b + half_b, &p.map_b[1], kk, col, pb, bar);
      } else if (B_MN) {
        const bool other = !A_MN && k >= second;  // of dx, which sums over both weights
        const CUtensorMap* map = other ? &p.map_b[1] : map_b;
        const int kb = other ? kk - (int)p.K1 : kk;
        mm_load_box<CTAS>(b, map, col, kb, pb, bar);
#pragma unroll
        for (int c = 1; c < kMmTileN / CTAS / 64; ++c)
          if (64 * c < cols) mm_load_box<CTAS>(b + c * 8192, map, col + 64 * c, kb, pb, bar);
      } else {
        mm_load_box<CTAS>(b, map_b, kk, col, pb, bar);
      }
    }
  }
  return done;
}

// A unit's products into the accumulators, by a whole warp of which one lane issues
// them: `chunk` steps into one half of them, the next into the other.  turn counts
// the chunks.  False where a wait gave up.
template <int EPI, int CTAS, bool A_MN>
__device__ __forceinline__ bool multiply_unit(const MmParams& p, uint32_t unit, const Place& at, Ring& ring,
                                              uint32_t& turn) {
  constexpr bool B_MN = EPI == MM_OUT;
  const uint32_t idesc = mm_idesc(A_MN, B_MN, kMmRows * CTAS, p.tn);
  const int stage_a = p.a_rows * kMmDepth * 2;
  uint32_t tile, split, left = steps_of(p, unit, tile, split), chunk = first_chunk(p, split);
  do {
    const uint32_t acc = turn & 1, d = at.tmem + acc * kMmTileN;
    if (!mm_warp_wait(at.acc_empty + 8 * acc, ((turn >> 1) & 1) ^ 1, at.guard)) return false;
    mm_fence_after();
    const uint32_t steps = left < chunk ? left : chunk;
    for (uint32_t i = 0; i < steps; ++i) {
      if (!mm_warp_wait(at.full + 8 * ring.stage, ring.round & 1, at.guard)) return false;
      mm_fence_after();
      const uint32_t a = at.stage0 + ring.stage * at.stage_bytes, free = at.empty + 8 * ring.stage;
      ring.next(at.stages);
      const uint64_t da = mm_desc(a, A_MN), db = mm_desc(a + stage_a, B_MN);
      if (!mm_elect()) continue;
#pragma unroll
      for (int j = 0; j < kMmDepth / 16; ++j)
        mm_mma<CTAS>(d, da + j * mm_desc_step(A_MN), db + j * mm_desc_step(B_MN), idesc, i > 0 || j > 0);
      mm_commit<CTAS>(free);
    }
    if (mm_elect()) mm_commit<CTAS>(at.acc_full + 8 * acc);
    ++turn;
    left -= steps;
    chunk = p.chunk;
  } while (left);
  return true;
}

// The accumulators of a turn may be summed into again, as far as this warp goes.
template <int CTAS>
__device__ __forceinline__ void release(const Place& at, uint32_t turn) {
  const uint32_t bar = at.acc_empty + 8 * (turn & 1);
  if (!mm_elect()) return;
  if (CTAS == 1)
    mm_bar_arrive(bar);
  else
    mm_bar_arrive_at(mm_of_first(bar));
}

// A warp's accumulators in tensor memory; zeros where nothing was summed.
struct TmemSource {
  uint32_t at;
  bool any;

  __device__ __forceinline__ void give(uint32_t (&r)[32], float (&v)[32]) const {
    mm_tmem_wait32(r);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = any ? __uint_as_float(r[j]) : 0.0f;
  }
  __device__ __forceinline__ void operator()(int c, float (&v)[32]) const {
    uint32_t r[32];
    mm_tmem_load(at + c, r);
    give(r, v);
  }
  // 16 columns from c, and 16 from d
  __device__ __forceinline__ void operator()(int c, int d, float (&v)[32]) const {
    uint32_t r[32];
    mm_tmem_load16(at + c, r);
    mm_tmem_load16(at + d, r + 16);
    give(r, v);
  }
};

// Chunks of a sum, added in registers.  The last one is not waited for here; the
// sum of the others is added to it in tensor memory by `finish`.  A warp's columns
// are two runs of 16 `groups` / 2 of them.
struct ChunkSum {
  float sum[8][16];

  // add: this chunk to the sum; else the sum to this chunk, in tensor memory
  template <bool ADD>
  __device__ __forceinline__ void take(uint32_t tmem, int run0, int run1, int groups) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (g >= groups) break;
      const uint32_t col = tmem + (g < groups / 2 ? run0 + 16 * g : run1 + 16 * (g - groups / 2));
      uint32_t r[16];
      mm_tmem_load16(col, r);
      mm_tmem_wait16(r);
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[g][j] += __uint_as_float(r[j]);
      if (!ADD) mm_tmem_store16(col, sum[g]);
    }
    if (!ADD) mm_tmem_stored();
  }
};

// What a warp has of a unit: 32 rows, and half of the columns, where a half has 64 of
// them.  In tensor memory these lie as two runs of `run` columns: of a gated tile,
// whose first half is gate's and whose second is up's, as many of each.  What the
// unit's sums go through in tensor memory is the warp's own runs and nothing else,
// since no barrier is between the warps.
struct Share {
  uint32_t tn, split, steps;
  int c0, c1, in_tile;
  int run0, run1, run;
  int64_t row0;
};
template <int EPI, int CTAS>
__device__ __forceinline__ Share share_of(const MmParams& p, uint32_t unit, const Place& at, int warp) {
  Share s;
  const int width = p.tn >= (EPI == MM_GATED ? 256 : 128) ? p.tn / 2 : p.tn;
  s.c0 = warp / 4 * width;
  s.c1 = s.c0 < p.tn ? s.c0 + width : s.c0;
  s.run = (s.c1 - s.c0) / 2;
  s.run0 = EPI == MM_GATED ? s.c0 / 2 : s.c0;
  s.run1 = EPI == MM_GATED ? p.tn / 2 + s.c0 / 2 : s.c0 + s.run;
  uint32_t tile, tm;
  s.steps = steps_of(p, unit, tile, s.split);
  tile_at(p, tile, tm, s.tn);
  s.in_tile = (int)at.rank * kMmRows + warp % 4 * 32;  // of tensor memory a warp reads a quarter
  s.row0 = (int64_t)tm * kMmRows * CTAS + s.in_tile;
  return s;
}

// A unit's epilogue once it is summed, or its sums left for the join; false where
// the wait gave up.
template <int EPI, int CTAS>
__device__ __forceinline__ bool finish_unit(const MmParams& p, uint32_t unit, const Place& at, uint32_t& turn, int warp,
                                            int lane, float* block) {
  constexpr int TILE_ROWS = kMmRows * CTAS;
  const Share mine = share_of<EPI, CTAS>(p, unit, at, warp);
  const int c0 = mine.c0, c1 = mine.c1, in_tile = mine.in_tile;
  const int64_t row0 = mine.row0;
  const uint32_t split = mine.split, tn = mine.tn, lanes = at.tmem + ((uint32_t)(warp % 4 * 32) << 16);
  uint32_t left = mine.steps;
  const MmRow row = mm_row<EPI>(p, row0, tn, lane);
  uint32_t chunk = first_chunk(p, split);
  if (left > chunk) {
    ChunkSum s = {};
    for (; left > chunk; left -= chunk, chunk = p.chunk, ++turn) {
      if (!mm_warp_wait(at.acc_full + 8 * (turn & 1), (turn >> 1) & 1, at.guard)) return false;
      mm_fence_after();
      s.take<true>(lanes + (turn & 1) * kMmTileN, mine.run0, mine.run1, mine.run / 8);
      mm_fence_before();
      __syncwarp();
      release<CTAS>(at, turn);
    }
    if (!mm_warp_wait(at.acc_full + 8 * (turn & 1), (turn >> 1) & 1, at.guard)) return false;
    mm_fence_after();
    s.take<false>(lanes + (turn & 1) * kMmTileN, mine.run0, mine.run1, mine.run / 8);
  } else {
    if (!mm_warp_wait(at.acc_full + 8 * (turn & 1), (turn >> 1) & 1, at.guard)) return false;
    mm_fence_after();
  }
  const TmemSource src = {lanes + (turn & 1) * kMmTileN, p.depth != 0};
  if (p.splits == 1) {
    mm_epilogue<EPI>(p, row0, tn, c0, c1, row, lane, block, src);
    mm_fence_before();
    __syncwarp();
    release<CTAS>(at, turn++);
    return true;
  }
  const int64_t rows = p.M < TILE_ROWS ? p.M : TILE_ROWS;
  float4* to = reinterpret_cast<float4*>(p.partial + (unit * rows + in_tile + lane) * p.tn);
  for (int i = 0; i < 2 * mine.run; i += 32) {
    const int c = i < mine.run ? mine.run0 + i : mine.run1 + i - mine.run;
    float x[32];
    src(c, x);
    if (row0 + lane < p.M) {
#pragma unroll
      for (int j = 0; j < 8; ++j) to[c / 4 + j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
  }
  mm_fence_before();
  __syncwarp();
  release<CTAS>(at, turn++);
  return true;
}

}  // namespace

// c[m, n] = sum over k of a[m, k] b[n, k], or of b[k, n] (MM_OUT), and the epilogue.
//
// Large products are bound by the tensor cores, whose rate the power limit sets in a
// long run.  Alone, us and PFLOP/s: the logits of 4096 x 32768 tokens and 4096 columns
// with what makes them e 551, 2.0; both gradients of those 1127, 1.95; 8192 x 128000 x
// 4096 to their log sum 4343, 2.0; the gated block of 16384 x 4096 x 11008 1490, 1.98.
// A tile of 256 x 256 by a pair reads 64 KB of operands for 512 cycles of products, a
// third less than two of 128 x 256; single CTAs are for products of less than a pair's
// rows, or with few tiles (the plan in products.cpp says which).  The eight warps of
// the epilogue have as long as the next tile's sum takes: with 64 steps and up
// they are hidden.
// Few rows are bound by the weight's bytes: 7 rows by 32000 x 4096 44, 6.0 TB/s; one
// row by two of 11008 x 4096 35, 5.1 TB/s, with 86 tiles for
// 152 SMs (in splits or narrower tiles it was no faster).
template <int EPI, int CTAS>
__global__ void __launch_bounds__(kMmThreads, 1) vc_mm(const __grid_constant__ MmLaunch all) {
  pdl_enter();
  extern __shared__ unsigned char raw[];
  __shared__ volatile int gave_up;
  __shared__ uint32_t tmem_at;
  constexpr bool TWO = EPI == MM_OUT;
  const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // the warp's, as the compiler sees it
  Place at;
  at.stage0 = (mm_smem(raw) + 1023) & ~1023u;  // of 128-byte swizzle atoms
  const uint32_t blocks = at.stage0 + kMmStageRoom;
  at.full = blocks + kMmEpilogueBytes;
  at.empty = at.full + 8 * kMmMaxStages;
  at.acc_full = at.empty + 8 * kMmMaxStages;
  at.acc_empty = at.acc_full + 16;
  at.drained = at.acc_empty + 16;
  at.rank = CTAS == 1 ? 0 : mm_rank();
  at.stages = all.stages;
  at.stage_bytes = all.stage_bytes;
  at.guard = {&gave_up, all.error_word};
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMmMaxStages; ++s) {
      mm_bar_init(at.full + 8 * s, 1);
      mm_bar_init(at.empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mm_bar_init(at.acc_full + 8 * s, 1);
      mm_bar_init(at.acc_empty + 8 * s, kMmEpilogueWarps * CTAS);
    }
    mm_bar_init(at.drained, 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmEpilogueWarps + 1) mm_tmem_alloc<CTAS>(mm_smem(&tmem_at));
  mm_fence_before();
  __syncthreads();
  if (CTAS > 1) mm_cluster_sync();
  mm_fence_after();
  at.tmem = __shfl_sync(~0u, tmem_at, 0);

  const uint32_t me = blockIdx.x / CTAS, of = gridDim.x / CTAS;
  Unit u;
  auto go_on = [&] { return !__any_sync(~0u, gave_up); };
  if (warp == kMmEpilogueWarps) {
    Ring ring;
    int64_t issued = 0;
    for (uint32_t n = 0; go_on() && unit_at<TWO>(all, me, of, n, u); ++n)
      issued += TWO && u.second ? load_unit<EPI, CTAS, true>(all.p[1], u.at, at, ring)
                                : load_unit<EPI, CTAS, false>(all.p[0], u.at, at, ring);
    if (!go_on() && at.rank == 0)  // copies cannot be called back: their memory has to stay until they have landed
      for (int64_t i = issued < at.stages ? 0 : issued - at.stages; i < issued; ++i)
        mm_warp_wait(at.full + 8 * (i % at.stages), (i / at.stages) & 1, at.guard, kMmDrainNs);
  } else if (warp == kMmEpilogueWarps + 1) {
    if (at.rank == 0) {
      Ring ring;
      uint32_t turn = 0;
      bool ok = true;
      for (uint32_t n = 0; ok && go_on() && unit_at<TWO>(all, me, of, n, u); ++n)
        ok = TWO && u.second ? multiply_unit<EPI, CTAS, true>(all.p[1], u.at, at, ring, turn)
                             : multiply_unit<EPI, CTAS, false>(all.p[0], u.at, at, ring, turn);
      if (!go_on()) {
        if (mm_elect()) mm_commit<CTAS>(at.drained);
        mm_warp_wait(at.drained, 0, at.guard, kMmDrainNs);
      }
    }
  } else {
    float* block = reinterpret_cast<float*>(raw + (blocks - mm_smem(raw))) + warp * kMmBlockWords;
    uint32_t turn = 0;
    for (uint32_t n = 0; unit_at<TWO>(all, me, of, n, u); ++n) {
      Unit next;
      if (EPI == MM_OUT)
        for (uint32_t ahead = n ? 1 : 0; ahead < 2 && unit_at<TWO>(all, me, of, n + ahead, next); ++ahead) {
          const MmParams& p = all.p[next.second];
          if (p.splits > 1 || (!p.accum_in && !p.base)) continue;
          const Share s = share_of<EPI, CTAS>(p, next.at, at, warp);
          mm_prefetch_added(p, s.row0, s.tn, s.c0, s.c1, lane);
        }
      if (!finish_unit<EPI, CTAS>(all.p[TWO && u.second], u.at, at, turn, warp, lane, block)) break;
    }
  }
  __syncwarp();
  mm_fence_before();
  __syncthreads();
  if (CTAS > 1) mm_cluster_sync();  // the other CTA's copies and products reach into this one's memory
  if (warp == kMmEpilogueWarps + 1) mm_tmem_free<CTAS>(at.tmem);
}

// The epilogue of tiles whose sums were cut: the splits' sums added in order, a
// warp for 32 columns of a row (MM_LSE: for a tile's), so that every load is a whole
// line.  Bound by those sums, which are still in L2, and by its launch: both gradients
// of 1000 x 5000 x 320 7.7 us, of 512 x 320 x 1280 5.3.
template <int EPI>
__global__ void __launch_bounds__(256) vc_mm_join_splits(const __grid_constant__ MmLaunch all) {
  pdl_enter();
  const bool second = blockIdx.x >= all.p[0].join_blocks;  // CTAs of p[0]'s come first
  const MmParams& p = all.p[second];
  const int lane = threadIdx.x % 32;
  const int tile_rows = p.tile_rows;
  const int64_t rows = p.M < tile_rows ? p.M : tile_rows;
  const int width = EPI == MM_GATED ? p.tn / 2 : p.tn, chunks = EPI == MM_LSE ? 1 : width / 32;
  const int64_t w = (int64_t)(blockIdx.x - (second ? all.p[0].join_blocks : 0)) * 8 + threadIdx.x / 32;
  const int chunk = (int)(w % chunks);
  const int64_t r = w / chunks % rows, tile = w / chunks / rows;
  if (tile >= (int64_t)p.tiles_m * p.tiles_n) return;
  uint32_t tm, tn;
  tile_at(p, (uint32_t)tile, tm, tn);
  const int64_t row = (int64_t)tm * tile_rows + r;
  if (row >= p.M) return;
  const float* from = p.partial + (tile * p.splits * rows + r) * p.tn;
  auto sum = [&](int c) {
    float x = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) x += from[s * rows * p.tn + c];
    return x;
  };
  const int c = chunk * 32 + lane;
  const int64_t col = (int64_t)tn * width + c;
  if constexpr (EPI == MM_OUT) {
    const MmOutRow to = mm_out_row(p, row);
    if (col >= p.N || to.row >= (p.M1 ? p.M2 : p.M)) return;
    float x = sum(c);
    const float scale = p.scale ? *p.scale : 1.0f;
    if (p.accum_scaled) x *= scale;
    if (p.accum_in) x += p.accum_in[row * p.accum_ld + col];
    if (p.accum_out) {
      p.accum_out[row * p.accum_ld + col] = x;
      return;
    }
    if (!p.accum_scaled) x *= scale;
    if (p.base) x += mm_load(p.base, p.out_f32, to.row * p.base_ld + col);
    mm_store(to.out, p.out_f32, to.row * to.ld + col, x);
  } else if constexpr (EPI == MM_LSE) {
    const int64_t t = mm_token(p.targets, p.idx64, row);
    const int64_t hit = t >= 0 && t < p.V ? t - p.token0 : -1;
    float v[kMmTileN / 32], top = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMmTileN / 32; ++i) {
      const int64_t at = (int64_t)tn * p.tn + i * 32 + lane;
      const bool in = i * 32 < p.tn && at < p.N;
      v[i] = in ? sum(i * 32 + lane) : -INFINITY;
      if (in && at == hit) p.picked[row] = v[i];
      top = fmaxf(top, v[i]);
    }
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float ref = mm_ref(top);
#pragma unroll
    for (int i = 0; i < kMmTileN / 32; ++i) s += mm_exp(v[i] - ref);
    for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
    if (lane == 0) p.part[(int64_t)tn * p.M + row] = make_float2(top, s);  // of the whole tile
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
    mm_store(p.out, p.out_f32, row * p.out_ld + col, mm_low(g) * (s * u));
  }
}

template <int CTAS>
static const void* kernel_of(MmEpilogue epilogue) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm<MM_LSE, CTAS>;
    case MM_ERROR:
      return (const void*)vc_mm<MM_ERROR, CTAS>;
    case MM_GATED:
      return (const void*)vc_mm<MM_GATED, CTAS>;
    default:
      return (const void*)vc_mm<MM_OUT, CTAS>;
  }
}

const void* mm_kernel(MmEpilogue epilogue, int ctas) {
  return ctas == 2 ? kernel_of<2>(epilogue) : kernel_of<1>(epilogue);
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
