// Embedding lookup and its gradient.
#include "device_common.cuh"
#include "layers_internal.h"

namespace vcoll {

namespace {

__device__ __forceinline__ int64_t token_at(const void* tokens, int idx64, int64_t i) {
  return idx64 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

template <typename T>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  return Elem<T>::widen1(static_cast<const typename Elem<T>::Bits*>(base)[i]);
}
template <typename T>
__device__ __forceinline__ void store1(void* base, int64_t i, float f) {
  static_cast<typename Elem<T>::Bits*>(base)[i] = Elem<T>::narrow1(f);
}

}  // namespace

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_embed(const __grid_constant__ EmbedParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < p.N; i += step) {
    const int64_t t = token_at(p.tokens, p.idx64, i);
    const bool inside = t >= 0 && t < p.V;
    for (int64_t c = lane; c < p.D; c += 32)
      store1<T>(p.out, i * p.out_ld + c,
                inside ? __fmul_rn(load1<T>(p.table, t * p.table_ld + c), p.scale) : 0.0f);
  }
}

// Stable LSD radix sort of the tokens' (key, position) pairs by one CTA.  Each
// warp owns a contiguous part of the array: it counts its digits, the counts
// are scanned over (digit, warp), and it walks its part again in order, the
// lanes of one digit taking the next places (match) in lane order.
__global__ void __launch_bounds__(kSortThreads) vc_embed_sort(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  constexpr int NW = kSortThreads / 32;
  extern __shared__ uint32_t cnt[];  // [digit][warp]
  __shared__ uint32_t wsum[NW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bins = 1 << p.bits;
  const int64_t per = ((p.N + NW - 1) / NW + 31) / 32 * 32;
  const int64_t lo = warp * per < p.N ? warp * per : p.N;
  const int64_t hi = lo + per < p.N ? lo + per : p.N;
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint32_t* key = p.key[(pass + 1) & 1];
    const uint32_t* pos = p.pos[(pass + 1) & 1];
    uint32_t* okey = p.key[pass & 1];
    uint32_t* opos = p.pos[pass & 1];
    const int shift = pass * p.bits;
    auto read = [&](int64_t i) -> uint32_t {
      if (pass) return key[i];
      const int64_t t = token_at(p.tokens, p.idx64, i);
      return t >= 0 && t < p.V ? (uint32_t)t : (uint32_t)p.V;
    };
    for (int b = threadIdx.x; b < bins * NW; b += kSortThreads) cnt[b] = 0;
    __syncthreads();
    for (int64_t i = lo + lane; i < hi; i += 32)
      atomicAdd(&cnt[((read(i) >> shift) & (bins - 1)) * NW + warp], 1u);
    __syncthreads();
    // exclusive scan over [digit][warp]: bins / NW' entries per thread
    const int each = bins * NW / kSortThreads;  // bins >= 32, so at least one
    uint32_t sum = 0;
    for (int k = 0; k < each; ++k) sum += cnt[threadIdx.x * each + k];
    uint32_t inc = sum;
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      uint32_t v = wsum[lane];
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += u;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    uint32_t run = inc - sum + (warp ? wsum[warp - 1] : 0u);
    for (int k = 0; k < each; ++k) {
      const uint32_t c = cnt[threadIdx.x * each + k];
      cnt[threadIdx.x * each + k] = run;
      run += c;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool in = i < hi;
      const uint32_t k = in ? read(i) : 0u;
      const uint32_t digit = (k >> shift) & (bins - 1);
      const uint32_t same = __match_any_sync(~0u, in ? digit : 0xFFFFFFFFu);
      const uint32_t before = __popc(same & ((1u << lane) - 1));
      uint32_t at = 0;
      if (in) at = cnt[digit * NW + warp] + before;
      __syncwarp();
      if (in && before == 0) cnt[digit * NW + warp] += __popc(same);
      __syncwarp();
      if (in) {
        okey[at] = k;
        opos[at] = pass ? pos[i] : (uint32_t)i;
      }
    }
    __syncthreads();
  }
}

// One warp per row of the table: its tokens' places in the sorted list by
// bisection, then the sum of their rows in order.
template <typename T, typename TO>
__global__ void __launch_bounds__(kRowThreads) vc_embed_grad(const __grid_constant__ EmbedGradParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kRowThreads / 32);
  const uint32_t* key = p.key[(p.passes + 1) & 1];
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  auto lower = [&](int64_t v) {
    int64_t a = 0, b = p.N;
    while (a < b) {
      const int64_t m = (a + b) >> 1;
      if ((int64_t)key[m] < v) a = m + 1;
      else b = m;
    }
    return a;
  };
  for (int64_t v = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); v < p.V; v += step) {
    const int64_t a = lower(v), b = lower(v + 1);
    if (a == b && p.in_place) continue;
    for (int64_t c = lane; c < p.D; c += 32) {
      float sum = 0.0f;
      for (int64_t k = a; k < b; ++k) sum += load1<T>(p.grad, (int64_t)pos[k] * p.grad_ld + c);
      sum *= p.scale;
      if (p.base) sum = load1<TO>(p.base, v * p.base_ld + c) + sum;
      store1<TO>(p.out, v * p.out_ld + c, sum);
    }
  }
}

const void* embed_kernel(int dtype) {
  return dtype == VCOLL_F32 ? (const void*)&vc_embed<float> : (const void*)&vc_embed<__nv_bfloat16>;
}
const void* embed_sort_kernel() { return (const void*)&vc_embed_sort; }
const void* embed_grad_kernel(int dtype, int table_dtype) {
  using B = __nv_bfloat16;
  if (dtype == VCOLL_F32)
    return table_dtype == VCOLL_F32 ? (const void*)&vc_embed_grad<float, float>
                                    : (const void*)&vc_embed_grad<float, B>;
  return table_dtype == VCOLL_F32 ? (const void*)&vc_embed_grad<B, float>
                                  : (const void*)&vc_embed_grad<B, B>;
}

}  // namespace vcoll
