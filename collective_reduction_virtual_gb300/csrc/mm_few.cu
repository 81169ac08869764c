// Products of a few fp32 rows, on the fp32 units.
//
// The tensor cores take fp32 operands as three bf16 parts, and laying a weight out
// as parts reads 4 bytes a value and writes 6 that are then read six times.  Where
// a weight meets a few rows only, reading it once bounds the product, and the
// fp32 units keep up with that to 16 rows (two operations a row for 4 bytes: 54
// TFLOP/s at 6.8 TB/s).  The small operand is in parts already, and is put
// together again in shared memory; the weight is read where it lies.
#include "mm_epilogue.cuh"

namespace vcoll {

namespace {

constexpr int kThreads = kMmFewThreads, kWarps = kThreads / 32;
constexpr int kColThreads = kMmFewColThreads, kColWarps = kColThreads / 32;
constexpr int kChunk = 512;  // places of a sum whose small operand is in shared memory
constexpr int kRows = 4;     // of the weight that a warp has in flight, and again as many

// Eight values of an operand in parts, from a multiple of 8 on; rows are as long.
__device__ __forceinline__ void from_parts(const MmOperand& o, int64_t row, int64_t col, float (&v)[8]) {
  const uint16_t* p = static_cast<const uint16_t*>(o.p) + row * o.ld + col;
  float q[3][8];
#pragma unroll
  for (int k = 0; k < 3; ++k) Elem<__nv_bfloat16>::widen(*reinterpret_cast<const uint4*>(p + k * o.plane), q[k]);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = q[0][j] + (q[1][j] + q[2][j]);
}

// A lane's four values: adjacent ones, 16 bytes at once, or without WIDE every 32nd,
// so that a warp reads 128 bytes in a row.
template <bool WIDE>
constexpr int kFirst = WIDE ? 4 : 1;  // places between lanes
template <bool WIDE>
constexpr int kNext = WIDE ? 1 : 32;  // and between a lane's four
// A value of what nothing writes meanwhile (FIXED: the weights), or of what the same
// kernel may write in place (base).
template <bool FIXED>
__device__ __forceinline__ float load1(const float* p) {
  return FIXED ? __ldg(p) : *p;
}
template <bool WIDE, bool FIXED>
__device__ __forceinline__ float4 load4(const float* p) {
  if (!WIDE) return make_float4(load1<FIXED>(p), load1<FIXED>(p + 32), load1<FIXED>(p + 64), load1<FIXED>(p + 96));
  const uint4 q = ld_stream(p);
  return make_float4(__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w));
}
// The same from place `at` of a row of `count` values, zeros past its end.
template <bool WIDE, bool FIXED>
__device__ __forceinline__ float4 load4_end(const float* row, int64_t at, int64_t count) {
  if (WIDE) return at < count ? load4<true, FIXED>(row + at) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  return make_float4(at < count ? load1<FIXED>(row + at) : 0.0f, at + 32 < count ? load1<FIXED>(row + at + 32) : 0.0f,
                     at + 64 < count ? load1<FIXED>(row + at + 64) : 0.0f,
                     at + 96 < count ? load1<FIXED>(row + at + 96) : 0.0f);
}

// The warp's sums of N values: those from lane * N / 32 on, N / 32 of them but one at
// least, in the lane's first.  In each step a lane gives half of what it has to the
// lane S away.
template <int S, int LEFT, int N>
__device__ __forceinline__ void scatter_sums(float (&v)[N], int lane) {
  const bool upper = lane & S;
  if constexpr (LEFT == 1) v[0] += __shfl_xor_sync(~0u, v[0], S);
#pragma unroll
  for (int j = 0; j < LEFT / 2; ++j) {
    const float give = upper ? v[j] : v[LEFT / 2 + j], keep = upper ? v[LEFT / 2 + j] : v[j];
    v[j] = keep + __shfl_xor_sync(~0u, give, S);
  }
  if constexpr (S > 1) scatter_sums<S / 2, LEFT / 2>(v, lane);
}

// A row of a tile's sums in shared memory.
struct FewSource {
  const float* row;
  __device__ __forceinline__ void operator()(int c, float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = row[c + j];
  }
  __device__ __forceinline__ void operator()(int c, int d, float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = row[c + j];
      v[16 + j] = row[d + j];
    }
  }
};

}  // namespace

// Rows of the small operand a times rows of the weight b: a CTA for all of a, ROWS
// at most, and 64 rows of b, four a warp, whose lanes go along the sum.  A warp's
// next loads are under way while it multiplies: four rows of 512 bytes, twice, is what
// keeps the memory busy at 16 warps.  Bound by the weight's bytes up to 4 rows
// (32000 x 4096, to the loss's tiles: 1 and 4 rows 98 us, 5.4 TB/s), above by the reads
// of xs that a warp needs for four rows' sums (8 rows 171, 16 205).
template <int EPI, int ROWS, bool WIDE>
__global__ void __launch_bounds__(kThreads) vc_mm_few_rows(const __grid_constant__ MmLaunch all) {
  pdl_enter();
  const MmParams& p = all.p[0];
  __shared__ __align__(16) float xs[ROWS][kChunk];
  __shared__ float sums[32 * 65];
  __shared__ float block[kMmBlockWords];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t tile_n = blockIdx.x;
  const bool second = EPI == MM_GATED && warp >= kWarps / 2;  // gate's rows, then as many of up's
  const MmOperand& b = p.b[second];
  const int64_t first = EPI == MM_GATED ? tile_n * 32 + warp % (kWarps / 2) * kRows : tile_n * 64 + warp * kRows;
  const float* w[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)  // rows past the end give columns that are not stored
    w[r] = static_cast<const float*>(b.p) + (first + r < b.rows ? first + r : b.rows - 1) * b.ld;
  constexpr int FIRST = kFirst<WIDE>, NEXT = kNext<WIDE>;
  float acc[kRows * ROWS] = {};
  float4 now[kRows], next[kRows];
  // a row's values from place k on, zeros past its end: its first one is read in their
  // place, since a load behind a condition would wait for the one before
  auto fetch = [&](const float* row, int64_t k) {
    const int64_t at = k + lane * FIRST;
    float4 v;
    if (WIDE) {
      const bool in = at < p.K;
      v = load4<true, true>(in ? row + at : row);
      if (!in) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
      const bool x = at < p.K, y = at + 32 < p.K, z = at + 64 < p.K, u = at + 96 < p.K;
      v = make_float4(__ldg(x ? row + at : row), __ldg(y ? row + at + 32 : row), __ldg(z ? row + at + 64 : row),
                      __ldg(u ? row + at + 96 : row));
      v.x = x ? v.x : 0.0f;
      v.y = y ? v.y : 0.0f;
      v.z = z ? v.z : 0.0f;
      v.w = u ? v.w : 0.0f;
    }
    return v;
  };
  if (p.K) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) next[r] = fetch(w[r], 0);
  }
  for (int64_t k0 = 0; k0 < p.K; k0 += kChunk) {
    for (int e = threadIdx.x; e < ROWS * (kChunk / 8); e += kThreads) {
      const int m = e / (kChunk / 8), k = e % (kChunk / 8) * 8;
      float v[8] = {};
      if (m < p.M && k0 + k < p.K) from_parts(p.a, m, k0 + k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) xs[m][k + j] = k0 + k + j < p.K ? v[j] : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kChunk && k0 + k < p.K; k += 128) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        now[r] = next[r];
        next[r] = fetch(w[r], k0 + k + 128);
      }
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        const float* at = &xs[m][k + lane * FIRST];
        const float4 x = WIDE ? *reinterpret_cast<const float4*>(at)
                              : make_float4(at[0], at[NEXT], at[2 * NEXT], at[3 * NEXT]);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          acc[r * ROWS + m] += (now[r].x * x.x + now[r].y * x.y) + (now[r].z * x.z + now[r].w * x.w);
      }
    }
    __syncthreads();
  }
  constexpr int EACH = kRows * ROWS / 32 > 0 ? kRows * ROWS / 32 : 1;
  scatter_sums<16, kRows * ROWS>(acc, lane);
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int at = (lane * kRows * ROWS >> 5) + j;  // r * ROWS + m
    sums[at % ROWS * 65 + warp * kRows + at / ROWS] = acc[j];
  }
  __syncthreads();
  if (warp) return;
  const FewSource src = {sums + lane * 65};
  mm_epilogue<EPI>(p, 0, tile_n, 0, p.tn, mm_row<EPI>(p, 0, tile_n, lane), lane, block, src);
}

// The small operand a times the weight b, which is taken transposed: a CTA for all
// rows, ROWS at most, 128 columns, four a lane, and a split of the sum, which its warps share.
// A split's sums go to vc_mm_join_splits.  Bound by the weight's bytes up to 8 rows:
// 32000 x 4096 with 1 row 83 us, 6.3 TB/s, with 8 102, with 16 180.
template <int ROWS, bool WIDE>
__global__ void __launch_bounds__(kColThreads, 2) vc_mm_few_cols(const __grid_constant__ MmLaunch all) {
  pdl_enter();
  const MmParams& p = all.p[0];
  constexpr int FLIGHT = ROWS == 16 ? 4 : 8;  // of the weight's rows that a warp has in flight, and again as many
  constexpr int CHUNK = 4096 / ROWS, FIRST = kFirst<WIDE>, NEXT = kNext<WIDE>;
  __shared__ float xs[CHUNK][ROWS];
  __shared__ float sums[ROWS][128];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t split = blockIdx.y;
  const int64_t col = (int64_t)blockIdx.x * 128 + lane * FIRST;
  const int64_t begin = p.K * split / p.splits & ~(int64_t)7;
  const int64_t end = split + 1 == p.splits ? p.K : p.K * (split + 1) / p.splits & ~(int64_t)7;
  const float *w0 = static_cast<const float*>(p.b[0].p), *w1 = static_cast<const float*>(p.b[1].p);
  const int64_t rows0 = p.b[0].rows, rows1 = p.b[1].rows, ld0 = p.b[0].ld, ld1 = p.b[1].ld;
  // the weight's rows at places k .. of the sum.  Columns past the end are not stored:
  // the last ones stand in for them, so that there is no condition between the loads.
  int64_t from[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) from[j] = WIDE ? (col < p.N ? col : p.N - 4) : col + 32 * j < p.N ? col + 32 * j : p.N - 1;
  float4 now[FLIGHT], next[FLIGHT];
  auto fetch = [&](int64_t k) {
    const bool second = k >= p.K1;
    const int64_t r = second ? k - p.K1 : k, rows = second ? rows1 : rows0, ld = second ? ld1 : ld0;
    const float* w = (second ? w1 : w0) + r * ld;
    if (k + FLIGHT <= end && r + FLIGHT <= rows) {
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i) {
        const float* q = w + i * ld;
        next[i] = WIDE ? load4<true, true>(q + from[0])
                       : make_float4(__ldg(q + from[0]), __ldg(q + from[1]), __ldg(q + from[2]), __ldg(q + from[3]));
      }
    } else {  // what pads a's first half has no row
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i)
        next[i] = load4_end<WIDE, true>(w + i * ld, col, k + i < end && r + i < rows ? p.N : 0);
    }
  };
  float acc[ROWS][4] = {};
  fetch(begin + warp * FLIGHT);
  for (int64_t k0 = begin; k0 < end; k0 += CHUNK) {
    for (int e = threadIdx.x; e < ROWS * (CHUNK / 8); e += kColThreads) {
      const int m = e % ROWS, k = e / ROWS * 8;
      float v[8] = {};
      if (m < p.M && k0 + k < end) from_parts(p.a, m, k0 + k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) xs[k + j][m] = k0 + k + j < end ? v[j] : 0.0f;
    }
    __syncthreads();
    for (int k = warp * FLIGHT; k < CHUNK && k0 + k < end; k += kColWarps * FLIGHT) {
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i) now[i] = next[i];
      // this warp's next rows: of this chunk, or its first of the next one
      const int64_t then = k0 + (k + kColWarps * FLIGHT < CHUNK ? k + kColWarps * FLIGHT : CHUNK + warp * FLIGHT);
      fetch(then);
#pragma unroll
      for (int i = 0; i < FLIGHT; ++i)
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
          const float x = xs[k + i][m];
          acc[m][0] += x * now[i].x;
          acc[m][1] += x * now[i].y;
          acc[m][2] += x * now[i].z;
          acc[m][3] += x * now[i].w;
        }
    }
    __syncthreads();
  }
  for (int q = 0; q < kColWarps; ++q) {  // one warp after the other: a fixed order
    if (warp == q) {
#pragma unroll
      for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float* at = &sums[m][lane * FIRST + j * NEXT];
          *at = q ? *at + acc[m][j] : acc[m][j];
        }
    }
    __syncthreads();
  }
  float* to = p.partial + ((int64_t)blockIdx.x * p.splits + split) * p.M * p.tn;
  for (int e = threadIdx.x; e < p.M * 128; e += kColThreads) to[e] = sums[0][e];
}

// The products of the columns of two small operands of a few rows: a CTA for
// 64 x 128 of the result, which it writes (and adds to base).  Bound by that up to
// 4 rows: 32000 x 4096 with 1 row 94 us, 5.6 TB/s, with 8 126, with 16 182.
template <bool WIDE>
__global__ void __launch_bounds__(kColThreads) vc_mm_few_outer(const __grid_constant__ MmLaunch all) {
  pdl_enter();
  const MmParams& p = all.p[1];
  __shared__ __align__(16) float es[kMmFewRows][64];
  __shared__ __align__(16) float xs[kMmFewRows][128];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t tiles = (p.N + 127) / 128;
  const int64_t row0 = blockIdx.x / tiles * 64, col0 = blockIdx.x % tiles * 128;
  const int K = (int)p.K;
  for (int e = threadIdx.x; e < K * 24; e += kColThreads) {
    const int k = e / 24, i = e % 24 * 8;  // 64 of es and 128 of xs; what is past their ends is not stored
    float v[8] = {};
    if (i < 64) {
      if (row0 + i < p.a.cols) from_parts(p.a, k, row0 + i, v);
    } else if (col0 + i - 64 < p.N) {
      from_parts(p.b[0], k, col0 + i - 64, v);
    }
    float* to = i < 64 ? &es[k][i] : &xs[k][i - 64];
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = v[j];
  }
  __syncthreads();
  float acc[8][4] = {};
#pragma unroll 2
  for (int k = 0; k < K; ++k) {
    const float4 x = WIDE ? *reinterpret_cast<const float4*>(&xs[k][lane * 4])
                          : make_float4(xs[k][lane], xs[k][lane + 32], xs[k][lane + 64], xs[k][lane + 96]);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float e = es[k][warp * 8 + r];
      acc[r][0] += e * x.x;
      acc[r][1] += e * x.y;
      acc[r][2] += e * x.z;
      acc[r][3] += e * x.w;
    }
  }
  const float scale = p.scale ? *p.scale : 1.0f;
  const int64_t col = col0 + (WIDE ? lane * 4 : lane);
  const MmOutRow to = mm_out_row(p, row0);
  const int64_t first = to.row + warp * 8, end = p.M1 ? p.M2 : p.M;
  float4 x[8];  // of base, all loads at once
#pragma unroll
  for (int r = 0; r < 8; ++r) x[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* base = static_cast<const float*>(p.base);
  if (base && first + 8 <= end && col0 + 128 <= p.N) {
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = load4<WIDE, false>(base + (first + r) * p.base_ld + col);
  } else if (base && first < end) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
      x[r] = load4_end<WIDE, false>(base + (first + r < end ? first + r : first) * p.base_ld, col, p.N);
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (first + r >= end) break;
    float* out = static_cast<float*>(to.out) + (first + r) * to.ld + col;
    const float4 y = make_float4(x[r].x + acc[r][0] * scale, x[r].y + acc[r][1] * scale, x[r].z + acc[r][2] * scale,
                                 x[r].w + acc[r][3] * scale);
    if (WIDE) {
      if (col < p.N) *reinterpret_cast<float4*>(out) = y;
    } else {
      if (col < p.N) out[0] = y.x;
      if (col + 32 < p.N) out[32] = y.y;
      if (col + 64 < p.N) out[64] = y.z;
      if (col + 96 < p.N) out[96] = y.w;
    }
  }
}

template <int ROWS, bool WIDE>
static const void* rows_kernel(MmEpilogue epilogue) {
  switch (epilogue) {
    case MM_LSE:
      return (const void*)vc_mm_few_rows<MM_LSE, ROWS, WIDE>;
    case MM_ERROR:
      return (const void*)vc_mm_few_rows<MM_ERROR, ROWS, WIDE>;
    case MM_GATED:
      return (const void*)vc_mm_few_rows<MM_GATED, ROWS, WIDE>;
    default:
      return (const void*)vc_mm_few_cols<ROWS, WIDE>;
  }
}
const void* mm_few_kernel(MmEpilogue epilogue, int rows, bool wide) {
  if (rows <= 4) return wide ? rows_kernel<4, true>(epilogue) : rows_kernel<4, false>(epilogue);
  if (rows <= 8) return wide ? rows_kernel<8, true>(epilogue) : rows_kernel<8, false>(epilogue);
  return wide ? rows_kernel<16, true>(epilogue) : rows_kernel<16, false>(epilogue);
}
const void* mm_few_outer_kernel(bool wide) {
  return wide ? (const void*)vc_mm_few_outer<true> : (const void*)vc_mm_few_outer<false>;
}

}  // namespace vcoll
