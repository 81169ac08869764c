// Layer norm, its gradient, and activations kept in 8 bits.
#include "device_common.cuh"
#include "layers_internal.h"

namespace vcoll {

namespace {

constexpr int kBlock8 = VCOLL_CHECKPOINT8_BLOCK;
constexpr float kTiny8 = 7.888609052210118e-31f;  // 2^-100

template <typename T>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  return Elem<T>::widen1(static_cast<const typename Elem<T>::Bits*>(base)[i]);
}
template <typename T>
__device__ __forceinline__ void store1(void* base, int64_t i, float f) {
  static_cast<typename Elem<T>::Bits*>(base)[i] = Elem<T>::narrow1(f);
}
// weights and biases, in either type; `none` where there is no such buffer
__device__ __forceinline__ float loadw(const void* w, int bf16, int64_t i, float none) {
  if (!w) return none;
  return bf16 ? load1<__nv_bfloat16>(w, i) : load1<float>(w, i);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
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

// The largest magnitude over a warp, NaN if any value is NaN.
__device__ __forceinline__ float warp_top(float a) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float b = __shfl_xor_sync(~0u, a, d);
    a = (b > a || b != b) ? b : a;
  }
  return a;
}
struct Scale8 {
  float scale, unit;
};
__device__ __forceinline__ Scale8 scale8(float top) {
  Scale8 s;
  if (!(top <= 3.402823466e38f)) {  // infinity or NaN
    s.scale = __uint_as_float(0x7FC00000u);
    s.unit = 0.0f;
  } else if (top < kTiny8) {
    s.scale = s.unit = 0.0f;
  } else {
    s.scale = __fdiv_rn(top, 127.0f);
    s.unit = __fdiv_rn(127.0f, top);
  }
  return s;
}
__device__ __forceinline__ int8_t code8(float x, const Scale8& s) {
  // a zero unit (zeros, or a block with a NaN or an infinity) gives code 0
  return s.unit == 0.0f ? (int8_t)0 : (int8_t)__float2int_rn(__fmul_rn(x, s.unit));
}

// One warp keeps one block of 128 columns; value(c) gives column c's value.
template <typename F>
__device__ __forceinline__ void keep_block(int64_t b, int64_t D, int8_t* codes, float* scale,
                                           F value) {
  const int lane = threadIdx.x & 31;
  float v[4], top = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t c = b * kBlock8 + k * 32 + lane;
    v[k] = c < D ? value(c) : 0.0f;
    const float a = fabsf(v[k]);
    top = (a > top || a != a) ? a : top;
  }
  const Scale8 s = scale8(warp_top(top));
  const int64_t end = (D + 15) / 16 * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t c = b * kBlock8 + k * 32 + lane;
    if (c < end) codes[c] = c < D ? code8(v[k], s) : (int8_t)0;
  }
  if (lane == 0) *scale = s.scale;
}

}  // namespace

// One CTA per row: the mean, the deviations' squares, then the outputs.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_norm(const __grid_constant__ NormParams p) {
  pdl_enter();
  __shared__ float red[kRowThreads / 32];
  for (int64_t i = blockIdx.x; i < p.N; i += gridDim.x) {
    const int64_t at = i * p.x_ld;
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) sum += load1<T>(p.x, at + c);
    const float mean = block_sum(sum, red) / (float)p.D;
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float d = load1<T>(p.x, at + c) - mean;
      sq += d * d;
    }
    const float rstd = rsqrtf(block_sum(sq, red) / (float)p.D + p.eps);
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
                h * loadw(p.weight, p.wbf16, c, 1.0f) + loadw(p.bias, p.wbf16, c, 0.0f));
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
__global__ void __launch_bounds__(kRowThreads) vc_norm_grad(const __grid_constant__ NormParams p) {
  pdl_enter();
  __shared__ float red[kRowThreads / 32];
  for (int64_t i = blockIdx.x; i < p.N; i += gridDim.x) {
    const float mean = p.x ? p.mean[i] : 0.0f, rstd = p.rstd[i];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float g = load1<T>(p.grad, i * p.grad_ld + c) * loadw(p.weight, p.wbf16, c, 1.0f);
      s1 += g;
      s2 += g * normal_at<T>(p, i, c, mean, rstd);
    }
    s1 = block_sum(s1, red) / (float)p.D;
    s2 = block_sum(s2, red) / (float)p.D;
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float g = load1<T>(p.grad, i * p.grad_ld + c) * loadw(p.weight, p.wbf16, c, 1.0f);
      store1<T>(p.y, i * p.y_ld + c, (g - s1 - normal_at<T>(p, i, c, mean, rstd) * s2) * rstd);
    }
  }
}

// One CTA per 32 columns: its warps sum every eighth row, then their sums.
// It runs before vc_norm_grad, which may write dx over grad or x.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_norm_wgrad(const __grid_constant__ NormParams p) {
  pdl_enter();
  constexpr int NW = kRowThreads / 32;
  __shared__ float sw[NW][32], sb[NW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float dw = 0.0f, db = 0.0f;
  if (c < p.D)
    for (int64_t i = warp; i < p.N; i += NW) {
      const float g = load1<T>(p.grad, i * p.grad_ld + c);
      dw += g * normal_at<T>(p, i, c, p.x ? p.mean[i] : 0.0f, p.rstd[i]);
      db += g;
    }
  sw[warp][lane] = dw;
  sb[warp][lane] = db;
  __syncthreads();
  if (warp || c >= p.D) return;
  dw = db = 0.0f;
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

// One warp per block of 128 columns.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_pack8(const __grid_constant__ PackParams p) {
  pdl_enter();
  const int64_t blocks = (p.D + kBlock8 - 1) / kBlock8;
  const int64_t step = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t k = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); k < p.N * blocks;
       k += step) {
    const int64_t i = k / blocks, b = k % blocks;
    keep_block(b, p.D, p.codes + i * p.codes_ld, p.scales + k,
               [&](int64_t c) { return load1<T>(p.x, i * p.x_ld + c); });
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) vc_unpack8(const __grid_constant__ PackParams p) {
  pdl_enter();
  const int64_t blocks = (p.D + kBlock8 - 1) / kBlock8;
  for (int64_t i = blockIdx.x; i < p.N; i += gridDim.x)
    for (int64_t c = threadIdx.x; c < p.D; c += kRowThreads) {
      const float h = (float)p.codes[i * p.codes_ld + c] * p.scales[i * blocks + c / kBlock8];
      store1<T>(p.out, i * p.x_ld + c,
                h * loadw(p.weight, p.wbf16, c, 1.0f) + loadw(p.bias, p.wbf16, c, 0.0f));
    }
}

#define VCOLL_BY_TYPE(fn) \
  (dtype == VCOLL_F32 ? (const void*)&fn<float> : (const void*)&fn<__nv_bfloat16>)
const void* norm_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm); }
const void* norm_grad_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm_grad); }
const void* norm_wgrad_kernel(int dtype) { return VCOLL_BY_TYPE(vc_norm_wgrad); }
const void* pack8_kernel(int dtype) { return VCOLL_BY_TYPE(vc_pack8); }
const void* unpack8_kernel(int dtype) { return VCOLL_BY_TYPE(vc_unpack8); }
#undef VCOLL_BY_TYPE

}  // namespace vcoll
