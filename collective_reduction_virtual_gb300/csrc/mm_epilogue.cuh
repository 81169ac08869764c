// What becomes of a tile of a product (MmEpilogue), a warp for 32 of its rows.
//
// The accumulators arrive as the tensor cores leave them: a lane holds one
// row, 32 columns at a time.  Sums along a row (MM_LSE) need no other lane.
// What is stored goes through a 32 x 33 block of shared memory, so that a warp
// writes 32 adjacent columns of one row after the other.
#pragma once

#include "device_common.cuh"
#include "mm_internal.h"

namespace vcoll {

constexpr int kMmPitch = 33;

__device__ __forceinline__ float mm_exp(float x) {  // e^x, to 2 ulp; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

__device__ __forceinline__ int64_t mm_token(const void* targets, int idx64, int64_t i) {
  return idx64 ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
}

__device__ __forceinline__ float mm_load(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : Elem<__nv_bfloat16>::widen1(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void mm_store(void* p, int f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = Elem<__nv_bfloat16>::narrow1(v);
}

// x as three bf16 values of 8 bits each, which together hold the 24 of an fp32
// mantissa.  Rounding to nearest leaves the remainders half as large as
// cutting off would; a value that rounds up to infinity is cut off.
__device__ __forceinline__ void mm_parts(float x, uint16_t (&q)[3]) {
  using B = Elem<__nv_bfloat16>;
  q[1] = q[2] = 0;
  q[0] = B::narrow1(x);
  if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u) return;  // no remainder
  if ((q[0] & 0x7F80u) == 0x7F80u) q[0] = (uint16_t)(__float_as_uint(x) >> 16);
  const float r1 = x - B::widen1(q[0]);
  q[1] = B::narrow1(r1);
  q[2] = B::narrow1(r1 - B::widen1(q[1]));
}

// The activations, g times a factor, and the factor's part in the derivative:
// act = g * s, act' = s + g * ds.  The exact gelu takes erfcf where g < 0, since
// 1 + erf loses the bits of a small result.
__device__ __forceinline__ void mm_act(int act, float g, float& s, float& ds) {
  if (act == VCOLL_SILU) {
    s = 1.0f / (1.0f + mm_exp(-g));
    ds = s * (1.0f - s);
  } else if (act == VCOLL_GELU) {
    s = 0.5f * erfcf(g * -0.70710678118654752f);
    ds = 0.39894228040143268f * mm_exp(-0.5f * g * g);
  } else {  // (1 + tanh(t)) / 2 = 1 / (1 + e^(-2 t))
    const float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    s = 1.0f / (1.0f + mm_exp(-c * (g + 0.044715f * g * g * g)));
    ds = s * (1.0f - s) * c * (1.0f + 0.134145f * g * g);
  }
}

__device__ __forceinline__ void mm_to_block(float* stage, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) stage[lane * kMmPitch + j] = v[j];
}

// f(r, value) for the rows r < rows of the warp's block, lane = column.
template <class F>
__device__ __forceinline__ void mm_by_rows(float* stage, int lane, const float (&v)[32], int rows,
                                           bool mine, F f) {
  mm_to_block(stage, lane, v);
  __syncwarp();
  if (mine) {
#pragma unroll 8
    for (int r = 0; r < rows; ++r) f(r, stage[r * kMmPitch + lane]);
  }
  __syncwarp();
}

// src(c, v): columns c .. c + 31 of this lane's row of the tile, called by the
// whole warp.  row0: the warp's first row of the result.
template <int EPI, class Source>
__device__ __forceinline__ void mm_epilogue(const MmParams& p, int64_t row0, int64_t tile_n,
                                            int lane, float* stage, Source src) {
  const int64_t row = row0 + lane;
  const int rows = (int)(p.M - row0 < 32 ? p.M - row0 : 32);  // < 1: only src is called
  float v[32];
  if constexpr (EPI == MM_OUT) {
    const float scale = p.scale ? *p.scale : 1.0f;
    for (int c = 0; c < p.tn; c += 32) {
      const int64_t col = tile_n * p.tn + c + lane;
      src(c, v);
      if (p.accum_out) {
        mm_by_rows(stage, lane, v, rows, col < p.N, [&](int r, float x) {
          const int64_t at = (row0 + r) * p.accum_ld + col;
          p.accum_out[at] = p.accum_in ? p.accum_in[at] + x : x;
        });
      } else {
        mm_by_rows(stage, lane, v, rows, col < p.N, [&](int r, float x) {
          if (p.accum_in) x += p.accum_in[(row0 + r) * p.accum_ld + col];
          x *= scale;
          if (p.base) x += mm_load(p.base, p.out_f32, (row0 + r) * p.base_ld + col);
          mm_store(p.out, p.out_f32, (row0 + r) * p.out_ld + col, x);
        });
      }
    }
  } else if constexpr (EPI == MM_LSE) {
    int64_t t = -1;
    if (lane < rows) t = mm_token(p.targets, p.idx64, row);
    const int64_t hit = t >= 0 && t < p.V ? t - p.token0 - tile_n * p.tn : -1;
    float m = -INFINITY, s = 0.0f;
    for (int c = 0; c < p.tn; c += 32) {
      src(c, v);
      const int64_t left = p.N - tile_n * p.tn - c;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (hit == c + j) p.picked[row] = v[j];
        if (j >= left) v[j] = -INFINITY;
        top = fmaxf(top, v[j]);
      }
      if (top > m) {
        s *= mm_exp(m - top);
        m = top;
      }
      const float ref = m == -INFINITY ? 0.0f : m;  // no difference of infinities
#pragma unroll
      for (int j = 0; j < 32; ++j) s += mm_exp(v[j] - ref);
    }
    if (lane < rows) p.part[tile_n * p.M + row] = make_float2(m, s);
  } else if constexpr (EPI == MM_ERROR) {
    int64_t t = -1;
    float lse = 0.0f, w = 0.0f;
    if (lane < rows) {
      t = mm_token(p.targets, p.idx64, row);
      lse = p.lse[row];
      w = p.dloss[row * p.dloss_step] / *p.scale;
    }
    const bool inside = t >= 0 && t < p.V;
    const int64_t hit = inside ? t - p.token0 - tile_n * p.tn : -1;
    uint16_t* error = static_cast<uint16_t*>(p.error);
    for (int c = 0; c < p.tn; c += 32) {
      const int64_t col = tile_n * p.tn + c + lane;
      src(c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float e = mm_exp(v[j] - lse);
        if (hit == c + j) e -= 1.0f;
        v[j] = inside ? e * w : 0.0f;
      }
      mm_by_rows(stage, lane, v, rows, col < p.N, [&](int r, float x) {
        const int64_t at = (row0 + r) * p.error_ld + col;
        if (p.parts == 1) {
          error[at] = Elem<__nv_bfloat16>::narrow1(x);
        } else {
          uint16_t q[3];
          mm_parts(x, q);
          for (int k = 0; k < 3; ++k) error[k * p.error_plane + at] = q[k];
        }
      });
    }
  } else {
    // in the layout by rows, so that a single row keeps all lanes busy
    const int half = p.tn / 2;
    float* other = stage + kMmBlockWords;
    for (int c = 0; c < half; c += 32) {
      const int64_t col = tile_n * half + c + lane;
      src(c, v);
      mm_to_block(stage, lane, v);
      src(half + c, v);
      mm_to_block(other, lane, v);
      __syncwarp();
      if (col < p.N) {
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
          const float g = stage[r * kMmPitch + lane], u = other[r * kMmPitch + lane];
          float s, ds;
          mm_act(p.act, g, s, ds);
          if (p.gate) mm_store(p.gate, p.out_f32, (row0 + r) * p.gate_ld + col, g);
          if (p.up) mm_store(p.up, p.out_f32, (row0 + r) * p.up_ld + col, u);
          mm_store(p.out, p.out_f32, (row0 + r) * p.out_ld + col, g * s * u);
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace vcoll
