// Layer norm and its gradient for rows of any width, the gradient's last sum,
// and 8-bit activations.
#include "norm_common.cuh"

namespace vcoll {

// ------------------------------------------------------ rows of any width
// For rows wider than a team of warps holds (norm_rows.cuh): a CTA per row
// that reads it again for each step, from L2 after the first; element by
// element, since such rows are rare and long enough to hide it.

namespace {

template <int K>
struct Sums {
  float v[K];
  __device__ __forceinline__ Sums() {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
  }
};
// each(i, part) for i = first, first + step, ... below end, kTerms of them with
// the same part, whose sums it adds to and which are then added up in sum: n terms
// in one chain are off by up to n u of the sum of their magnitudes, these by
// kTerms + n / kTerms (u = 2^-24).  Eight terms' loads go out together: 20000 x
// 16400 fp32 650 us forward and 1146 backward (one chain: 620 and 1575).
template <int K, typename F>
__device__ __forceinline__ Sums<K> long_sums(int64_t first, int64_t end, int step, F each) {
  constexpr int kTerms = 64;
  Sums<K> sum;
  for (int64_t i = first; i < end;) {
    Sums<K> part;
    const int64_t stop = min(end, i + (int64_t)kTerms * step);
#pragma unroll 8
    for (; i < stop; i += step) each(i, part.v);
#pragma unroll
    for (int k = 0; k < K; ++k) sum.v[k] += part.v[k];
  }
  return sum;
}

// Sum over the CTA, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f);
}

// One warp keeps one block of 128 columns; value(c) gives column c's value.
template <typename F>
__device__ __forceinline__ void keep_block(int64_t b, int64_t D, int8_t* codes, float* scale,
                                           F value) {
  const int lane = threadIdx.x & 31;
  float v[1][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t c = b * kBlock8 + k * 32 + lane;
    v[0][k] = c < D ? value(c) : 0.0f;
  }
  // as fp32 in single elements: 4 groups of 32 columns, one block
  const int64_t left = D - b * kBlock8;
  keep8<float, 1, 1>(v, 0, lane, left < kBlock8 ? (int)left : kBlock8, codes + b * kBlock8, scale);
}

}  // namespace

// One CTA per row: the mean, the deviations' squares, then the outputs.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_norm_wide(const __grid_constant__ NormParams p) {
  pdl_enter();
  __shared__ float red[kRowThreads / 32];
  for (int64_t i = blockIdx.x; i < p.N; i += gridDim.x) {
    const int64_t at = i * p.x_ld;
    const Sums<1> sum = long_sums<1>(threadIdx.x, p.D, kRowThreads,
                                     [&](int64_t c, float* s) { *s += load1<T>(p.x, at + c); });
    const float mean = block_sum(sum.v[0], red) / (float)p.D;
    const Sums<1> sq = long_sums<1>(threadIdx.x, p.D, kRowThreads, [&](int64_t c, float* s) {
      const float d = load1<T>(p.x, at + c) - mean;
      *s += d * d;
    });
    const float rstd = rsqrtf(block_sum(sq.v[0], red) / (float)p.D + p.eps);
    if (p.codes) {
      const int64_t blocks = (p.D + kBlock8 - 1) / kBlock8;
      for (int64_t b = threadIdx.x >> 5; b < blocks; b += kRowThreads / 32)
        keep_block(b, p.D, p.codes + i * p.codes_ld, p.scales + i * blocks + b,
                   [&](int64_t c) { return (load1<T>(p.x, at + c) - mean) * rstd; });
      __syncthreads();  // y may be x
    }
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float h = (load1<T>(p.x, at + c) - mean) * rstd;
      store1<T>(p.y, i * p.y_ld + c,
                h * load_weight(p.weight, p.wbf16, c, 1.0f) + load_weight(p.bias, p.wbf16, c, 0.0f));
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[i] = mean;
      if (p.rstd) p.rstd[i] = rstd;
    }
  }
}

namespace {
// h of row i, column c: from x and the row's statistics, or from the codes.
template <typename T>
__device__ __forceinline__ float normal_at(const NormParams& p, int64_t i, int64_t c, float mean,
                                           float rstd) {
  if (p.x) return (load1<T>(p.x, i * p.x_ld + c) - mean) * rstd;
  const int64_t blocks = (p.D + kBlock8 - 1) / kBlock8;
  return (float)p.codes[i * p.codes_ld + c] * p.scales[i * blocks + c / kBlock8];
}
}  // namespace

// One CTA per row: the two sums of the row, then dx.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_norm_grad_wide(const __grid_constant__ NormParams p) {
  pdl_enter();
  __shared__ float red[kRowThreads / 32];
  for (int64_t i = blockIdx.x; i < p.N; i += gridDim.x) {
    const float mean = p.x ? p.mean[i] : 0.0f, rstd = p.rstd[i];
    const Sums<2> sum = long_sums<2>(threadIdx.x, p.D, kRowThreads, [&](int64_t c, float* s) {
      const float g = load1<T>(p.grad, i * p.grad_ld + c) * load_weight(p.weight, p.wbf16, c, 1.0f);
      s[0] += g;
      s[1] += g * normal_at<T>(p, i, c, mean, rstd);
    });
    const float s1 = block_sum(sum.v[0], red) / (float)p.D;
    const float s2 = block_sum(sum.v[1], red) / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float g = load1<T>(p.grad, i * p.grad_ld + c) * load_weight(p.weight, p.wbf16, c, 1.0f);
      store1<T>(p.y, i * p.y_ld + c, (g - s1 - normal_at<T>(p, i, c, mean, rstd) * s2) * rstd);
    }
  }
}

// One CTA per 32 columns: its warps sum every eighth row, then their sums.
// It runs before vc_norm_grad_wide, which may write dx over grad or x.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_norm_wgrad_wide(const __grid_constant__ NormParams p) {
  pdl_enter();
  constexpr int NW = kRowThreads / 32;
  __shared__ float sw[NW][32], sb[NW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const Sums<2> sum = long_sums<2>(warp, c < p.D ? p.N : 0, NW, [&](int64_t i, float* s) {
    const float g = load1<T>(p.grad, i * p.grad_ld + c);
    s[0] += g * normal_at<T>(p, i, c, p.x ? p.mean[i] : 0.0f, p.rstd[i]);
    s[1] += g;
  });
  sw[warp][lane] = sum.v[0];
  sb[warp][lane] = sum.v[1];
  __syncthreads();
  if (warp || c >= p.D) return;
  float dw = 0.0f, db = 0.0f;
  for (int k = 0; k < NW; ++k) {
    dw += sw[k][lane];
    db += sb[k][lane];
  }
  if (p.wbf16) {
    if (p.dweight) store1<__nv_bfloat16>(p.dweight, c, dw);
    if (p.dbias) store1<__nv_bfloat16>(p.dbias, c, db);
  } else {
    if (p.dweight) store1<float>(p.dweight, c, dw);
    if (p.dbias) store1<float>(p.dbias, c, db);
  }
}

// ------------------------------------------ the gradient's sum over the CTAs

// part[cta][2][D] summed over the CTAs: a CTA per 32 columns of one of the
// two; its warps take every 32nd row, and each adds up one column's sums.  304
// rows of 4096 columns: 5 us, from L2.
__global__ void __launch_bounds__(1024) vc_norm_wsum(const __grid_constant__ NormParams p) {
  pdl_enter();
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  void* out = blockIdx.y ? p.dbias : p.dweight;
  if (!out) return;
  float s = 0.0f;
  if (c < p.D) {
    const float* from = p.part + blockIdx.y * p.D + c;
#pragma unroll 8
    for (int k = warp; k < p.parts; k += 32) s += from[(int64_t)k * 2 * p.D];
  }
  sum[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sum[lane][warp]);  // column `warp` of this CTA's
  const int64_t col = (int64_t)blockIdx.x * 32 + warp;
  if (lane || col >= p.D) return;
  if (p.wbf16) store1<__nv_bfloat16>(out, col, s);
  else store1<float>(out, col, s);
}

// ------------------------------------------------------- 8-bit activations
// A warp takes kPackChunks chunks of 32 * E columns of a row, all of their
// loads in flight.  Bound by HBM: 9001 x 2052 fp32 kept and restored in 30 us,
// 6.3 TB/s; 32768 x 4096 bf16 67 and 65 us, 6.0 and 6.2 TB/s.

template <typename T, int A>
__global__ void __launch_bounds__(kRowThreads) vc_pack8(const __grid_constant__ PackParams p) {
  pdl_enter();
  constexpr int R = kPackChunks;
  using P = Lanes<T, A, R>;
  constexpr int E = P::E;
  const int D = (int)p.D;
  const RowPiece piece((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), p.pieces);
  const int64_t i = piece.row;
  if (i >= p.N) return;
  const int col = (int)piece.piece * P::kColumns, c = col + P::first(threadIdx.x & 31);
  uint4 raw[R];
  if (D - col >= P::kColumns) P::template load<true>(raw, elem_at<T>(p.x, i * p.x_ld), c, D);
  else P::template load<false>(raw, elem_at<T>(p.x, i * p.x_ld), c, D);
  float f[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) Elem<T>::widen(raw[r], f[r]);
  keep8<T, A, R>(f, col, c, D, p.codes + i * p.codes_ld, p.scales + i * ((D + kBlock8 - 1) / kBlock8));
}

template <typename T, int A>
__global__ void __launch_bounds__(kRowThreads) vc_unpack8(const __grid_constant__ PackParams p) {
  pdl_enter();
  constexpr int R = kPackChunks;
  using P = Lanes<T, A, R>;
  using Q = Lanes<T, A, 1>;  // one chunk
  constexpr int E = P::E;
  const int D = (int)p.D;
  const RowPiece piece((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), p.pieces);
  const int64_t i = piece.row;
  if (i >= p.N) return;
  char* out = elem_at<T>(p.out, i * p.x_ld);
  const int8_t* codes = p.codes + i * p.codes_ld;
  const float* scales = p.scales + i * ((D + kBlock8 - 1) / kBlock8);
  const int col = (int)piece.piece * P::kColumns, c = col + P::first(threadIdx.x & 31);
  auto group = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    uint32_t word[R][2];
    float scale[R][E / 4];  // of each four elements
#pragma unroll
    for (int r = 0; r < R; ++r) {
      word[r][0] = word[r][1] = 0u;
      if constexpr (A == E) {
        scale[r][0] = 0.0f;
        if (P::template inside<FULL>(r, 0, c, D)) {
          const int at = c + P::offset(r, 0);
          scale[r][0] = scales[at / kBlock8];
          if constexpr (E == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(codes + at));
            word[r][0] = v.x;
            word[r][1] = v.y;
          } else {
            word[r][0] = __ldcs(reinterpret_cast<const uint32_t*>(codes + at));
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool in = P::template inside<FULL>(r, e, c, D);
          if (in) word[r][e / 4] |= (uint32_t)(uint8_t)codes[c + P::offset(r, e)] << (8 * (e % 4));
          if (e % 4 == 0) scale[r][e / 4] = in ? scales[(c + P::offset(r, e)) / kBlock8] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int cr = c + r * 32 * E;
      float f[1][E];
#pragma unroll
      for (int e = 0; e < E; e += 2)
        code_values(word[r][e / 4], e % 4, scale[r][A == E ? 0 : e / 4], f[0][e], f[0][e + 1]);
      Q::template affine<FULL>(p.weight, p.bias, p.wbf16, cr, D, f);
      Q::template store<FULL>(out, cr, D, f);
    }
  };
  if (D - col >= P::kColumns) group(Bool<true>());
  else group(Bool<false>());
}

// Narrow rows, kNarrowRows of each group of G lanes in flight (100000 x 64 bf16:
// 5.5 and 5.6 us; a warp per row took 34 and 39).
template <typename T, int A, int G>
__global__ void __launch_bounds__(kRowThreads) vc_pack8_narrow(const __grid_constant__ PackParams p) {
  pdl_enter();
  const Group<T, A, G> g;
  constexpr int E = kLane<T>, U = kNarrowRows, S = 32 / G;
  const int D = (int)p.D;
  const int64_t first = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * (U * S) + g.sub;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * S;
    raw[u] = g.load(elem_at<T>(p.x, i * p.x_ld), D, i < p.N);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * S;
    float f[E];
    Elem<T>::widen(raw[u], f);
    g.keep(f, D, i < p.N, p.codes + i * p.codes_ld, p.scales + i * ((D + kBlock8 - 1) / kBlock8));
  }
}
template <typename T, int A, int G>
__global__ void __launch_bounds__(kRowThreads) vc_unpack8_narrow(const __grid_constant__ PackParams p) {
  pdl_enter();
  const Group<T, A, G> g;
  constexpr int E = kLane<T>, U = kNarrowRows, S = 32 / G;
  const int D = (int)p.D;
  const int64_t first = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * (U * S) + g.sub;
  float f[U][E], w[E], b[E];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * S;
    g.kept(p.codes + i * p.codes_ld, p.scales + i * ((D + kBlock8 - 1) / kBlock8), D, i < p.N, f[u]);
  }
  g.weights(p.weight, p.wbf16, D, 1.0f, w);
  g.weights(p.bias, p.wbf16, D, 0.0f, b);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * S;
    if (i >= p.N) return;
    if (p.weight || p.bias)
#pragma unroll
      for (int e = 0; e < E; e += 2)
        fma2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], w[e], w[e + 1], b[e], b[e + 1]);
    g.store(elem_at<T>(p.out, i * p.x_ld), D, f[u]);
  }
}

#define VCOLL_BY_TYPE(fn) \
  (dtype == VCOLL_F32 ? (const void*)&fn<float> : (const void*)&fn<__nv_bfloat16>)
#define VCOLL_BY_ACCESS(fn)                                                                \
  (dtype == VCOLL_F32 ? access == 4 ? (const void*)&fn<float, 4> : (const void*)&fn<float, 1> \
   : access == 8      ? (const void*)&fn<__nv_bfloat16, 8>                                 \
   : access == 2      ? (const void*)&fn<__nv_bfloat16, 2>                                 \
                      : (const void*)&fn<__nv_bfloat16, 1>)
const void* norm_wide_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm_wide); }
const void* norm_grad_wide_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm_grad_wide); }
const void* norm_wgrad_wide_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm_wgrad_wide); }
const void* norm_wsum_kernel() { return (const void*)&vc_norm_wsum; }
const void* pack8_kernel(int dtype, int access) { return VCOLL_BY_ACCESS(vc_pack8); }
const void* unpack8_kernel(int dtype, int access) { return VCOLL_BY_ACCESS(vc_unpack8); }

namespace {
template <typename T, int A>
const void* narrow(int lanes, bool unpack) {
  if (lanes == 8) return unpack ? (const void*)&vc_unpack8_narrow<T, A, 8> : (const void*)&vc_pack8_narrow<T, A, 8>;
  if (lanes == 16) return unpack ? (const void*)&vc_unpack8_narrow<T, A, 16> : (const void*)&vc_pack8_narrow<T, A, 16>;
  return unpack ? (const void*)&vc_unpack8_narrow<T, A, 32> : (const void*)&vc_pack8_narrow<T, A, 32>;
}
}  // namespace
const void* pack8_narrow_kernel(int dtype, int access, int lanes, bool unpack) {
  if (dtype == VCOLL_F32) return access == 4 ? narrow<float, 4>(lanes, unpack) : narrow<float, 1>(lanes, unpack);
  return access == 8   ? narrow<__nv_bfloat16, 8>(lanes, unpack)
         : access == 2 ? narrow<__nv_bfloat16, 2>(lanes, unpack)
                       : narrow<__nv_bfloat16, 1>(lanes, unpack);
}
#undef VCOLL_BY_TYPE
#undef VCOLL_BY_ACCESS

}  // namespace vcoll
