// Products with the element-wise part of an operator as their epilogue.
//
// The simple form: a CTA of 256 threads for a tile of 128 x 64, both operands
// through shared memory 16 places of the sum at a time, fp32 multiply-adds.
// Correct for every size and stride, and bound by the fp32 units.
#include "mm_epilogue.cuh"

namespace vcoll {

namespace {

constexpr int kDepth = 16;

// A block of `tile` x kDepth of an operand, from row (of the result) i0 and
// place k0 of the sum; zeros outside.
template <bool MN>
__device__ __forceinline__ void load_block(const MmOperand& o, int part, int64_t i0, int tile,
                                           int64_t k0, float* to) {
  const uint16_t* p = static_cast<const uint16_t*>(o.p) + part * o.plane;
  for (int e = threadIdx.x; e < tile * kDepth; e += kMmSimpleThreads) {
    const int i = MN ? e % tile : e / kDepth, k = MN ? e / tile : e % kDepth;
    const int64_t r = MN ? k0 + k : i0 + i, c = MN ? i0 + i : k0 + k;
    to[k * (tile + 1) + i] = r < o.rows && c < o.cols ? Elem<__nv_bfloat16>::widen1(p[r * o.ld + c]) : 0.0f;
  }
}

}  // namespace

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kMmSimpleThreads) vc_mm_simple(const __grid_constant__ MmParams p) {
  pdl_enter();
  constexpr int TN = kMmSimpleTileN;
  __shared__ float a[kDepth * (kMmTileM + 1)], b[kDepth * (TN + 1)];
  __shared__ float sums[kMmTileM * (TN + 1)];
  __shared__ float stage[4 * kMmStageWords];
  const int64_t tile_m = blockIdx.x % p.tiles_m, tile_n = blockIdx.x / p.tiles_m;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[8][4] = {};
  const int pairs = mm_pairs(p.parts);
  for (int q = 0; q < pairs; ++q) {
    const int pa = mm_pair_a(pairs, q), pb = mm_pair_b(pairs, q);
    for (int64_t k0 = 0; k0 < p.K; k0 += kDepth) {
      const bool second = k0 >= p.K1;
      load_block<A_MN>(p.a, pa, tile_m * kMmTileM, kMmTileM, k0, a);
      if (p.b_halves) {
        for (int h = 0; h < 2; ++h) {
          // columns h * TN / 2 .. of the block
          const MmOperand& o = p.b[h];
          for (int e = threadIdx.x; e < TN / 2 * kDepth; e += kMmSimpleThreads) {
            const int i = e / kDepth, k = e % kDepth;
            const int64_t r = tile_n * (TN / 2) + i, c = k0 + k;
            b[k * (TN + 1) + h * (TN / 2) + i] =
                r < o.rows && c < o.cols
                    ? Elem<__nv_bfloat16>::widen1(static_cast<const uint16_t*>(o.p)[pb * o.plane + r * o.ld + c])
                    : 0.0f;
          }
        }
      } else {
        load_block<B_MN>(p.b[second], pb, tile_n * TN, TN, second ? k0 - p.K1 : k0, b);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kDepth; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] += a[k * (kMmTileM + 1) + ty + 16 * i] * b[k * (TN + 1) + tx + 16 * j];
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[(ty + 16 * i) * (TN + 1) + tx + 16 * j] = acc[i][j];
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp < 4) {
    const float* row = sums + (warp * 32 + lane) * (TN + 1);
    mm_epilogue<EPI>(p, tile_m * kMmTileM + warp * 32, tile_n, lane, stage + warp * kMmStageWords,
                     [&](int c, float (&v)[32]) {
#pragma unroll
                       for (int j = 0; j < 32; ++j) v[j] = row[c + j];
                     });
  }
}

const void* mm_simple_kernel(int epilogue, bool a_mn) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm_simple<MM_LSE, false, false>;
    case MM_ERROR:
      return (const void*)vc_mm_simple<MM_ERROR, false, false>;
    case MM_GATED:
      return (const void*)vc_mm_simple<MM_GATED, false, false>;
    default:
      return a_mn ? (const void*)vc_mm_simple<MM_OUT, true, true> : (const void*)vc_mm_simple<MM_OUT, false, true>;
  }
}

}  // namespace vcoll
