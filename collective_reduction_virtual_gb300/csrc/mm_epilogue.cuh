// What becomes of a tile of a product (MmEpilogue), a warp for 32 of its rows.
//
// The accumulators arrive as the tensor cores leave them: a lane holds a row,
// 32 columns at a time.  What goes along a row (exponentials, activations, a
// row's maximum and sum) is done there, in registers.  What is stored goes
// through a 32 x 33 block of shared memory, so that a warp writes 128 adjacent
// bytes of one row after the other.
#pragma once

#include "device_common.cuh"
#include "mm_internal.h"

namespace vcoll {

__device__ __forceinline__ float mm_exp2(float x) {  // 2 ulp; 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kMmLog2e = 1.4426950408889634f;
__device__ __forceinline__ float mm_exp(float x) { return mm_exp2(x * kMmLog2e); }
__device__ __forceinline__ float mm_rcp(float x) {  // 1 ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int64_t mm_token(const void* targets, int idx64, int64_t i) {
  return idx64 ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
}

__device__ __forceinline__ float mm_load(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : Elem<__nv_bfloat16>::widen1(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ uint16_t mm_narrow(float x) {  // a NaN gives the conversion's
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<const uint16_t*>(&h);
}
__device__ __forceinline__ uint32_t mm_narrow2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void mm_store(void* p, int f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = mm_narrow(v);
}

// x as three bf16 values of 8 bits each, which together hold the 24 of an fp32
// mantissa.  Rounding to nearest leaves the remainders half as large as
// cutting off would; a value that rounds up to infinity is cut off.
__device__ __forceinline__ void mm_parts(float x, uint16_t (&q)[3]) {
  using B = Elem<__nv_bfloat16>;
  q[1] = q[2] = 0;
  q[0] = mm_narrow(x);
  if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u) return;  // no remainder
  if ((q[0] & 0x7F80u) == 0x7F80u) q[0] = (uint16_t)(__float_as_uint(x) >> 16);
  const float r1 = x - B::widen1(q[0]);
  q[1] = mm_narrow(r1);
  q[2] = mm_narrow(r1 - B::widen1(q[1]));
}

// The activations, g times a factor, and the factor's part in the derivative:
// act = g * s, act' = s + g * ds.  The exact gelu takes erfcf where g < 0, since
// 1 + erf loses the bits of a small result.
__device__ __forceinline__ void mm_act(int act, float g, float& s, float& ds) {
  if (act == VCOLL_SILU) {
    s = mm_rcp(1.0f + mm_exp(-g));
    ds = s * (1.0f - s);
  } else if (act == VCOLL_GELU) {
    s = 0.5f * erfcf(g * -0.70710678118654752f);
    ds = 0.39894228040143268f * mm_exp(-0.5f * g * g);
  } else {  // (1 + tanh(t)) / 2 = 1 / (1 + e^(-2 t))
    const float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    s = mm_rcp(1.0f + mm_exp(-c * (g + 0.044715f * g * g * g)));
    ds = s * (1.0f - s) * c * (1.0f + 0.134145f * g * g);
  }
}

template <int ACT>
__device__ __forceinline__ void mm_gate(float (&g)[32], const float (&u)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float s, ds;
    mm_act(ACT, g[j], s, ds);
    g[j] *= s * u[j];
  }
}

// Where a row of the result goes.
struct MmOutRow {
  void* out;
  int64_t ld, row;  // within out
};
__device__ __forceinline__ MmOutRow mm_out_row(const MmParams& p, int64_t row) {
  const bool second = p.M1 && row >= p.M1;
  return {second ? p.out2 : p.out, second ? p.out2_ld : p.out_ld, second ? row - p.M1 : row};
}
// of 32 rows from row0 on: those that are the result's
__device__ __forceinline__ int mm_rows(const MmParams& p, int64_t row0) {
  const int64_t end = !p.M1 ? p.M : row0 >= p.M1 ? p.M1 + p.M2 : p.M2;
  return (int)(end - row0 < 32 ? end - row0 : 32);
}

// A warp's block by rows: for the rows r < rows, x = load(r, word) eight at a
// time, then store(r, x).
template <class Load, class Store>
__device__ __forceinline__ void mm_by_rows(const uint32_t* block, int lane, int rows, bool mine, Load load,
                                           Store store) {
  __syncwarp();
  if (mine) {
    for (int r = 0; r < rows; r += 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i < rows) x[i] = load(r + i, block[(r + i) * kMmPitch + lane]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i < rows) store(r + i, x[i]);
    }
  }
  __syncwarp();
}

// 64 columns of bf16, two to a word, into rows that allow 4-byte stores.
__device__ __forceinline__ void mm_store_pairs(uint32_t* block, int lane, const float (&a)[32],
                                               const float (&b)[32], int rows, uint16_t* to, int64_t ld,
                                               int64_t left) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    block[lane * kMmPitch + j] = mm_narrow2(a[2 * j], a[2 * j + 1]);
    block[lane * kMmPitch + 16 + j] = mm_narrow2(b[2 * j], b[2 * j + 1]);
  }
  __syncwarp();
  uint16_t* at = to + 2 * lane;
  if (2 * lane + 1 < left) {
    if (rows >= 32) {
#pragma unroll
      for (int r = 0; r < 32; ++r)
        *reinterpret_cast<uint32_t*>(at + r * ld) = block[r * kMmPitch + lane];
    } else {
      for (int r = 0; r < rows; ++r)
        *reinterpret_cast<uint32_t*>(at + r * ld) = block[r * kMmPitch + lane];
    }
  } else if (2 * lane < left) {
    for (int r = 0; r < rows; ++r) at[r * ld] = (uint16_t)block[r * kMmPitch + lane];
  }
  __syncwarp();
}

// 32 columns, a store for each value.
__device__ __forceinline__ void mm_store_each(uint32_t* block, int lane, const float (&v)[32], int rows,
                                              void* to, int f32, int64_t at, int64_t ld, int64_t left) {
#pragma unroll
  for (int j = 0; j < 32; ++j) block[lane * kMmPitch + j] = __float_as_uint(v[j]);
  mm_by_rows(
      block, lane, rows, lane < left, [](int, uint32_t w) { return __uint_as_float(w); },
      [&](int r, float x) { mm_store(to, f32, at + r * ld + lane, x); });
}

// 64 columns of a matrix of the operator's type.
__device__ __forceinline__ void mm_store_64(uint32_t* block, int lane, const float (&a)[32], const float (&b)[32],
                                            int rows, void* to, int f32, int pairs, int64_t row, int64_t ld,
                                            int64_t col, int64_t cols) {
  const int64_t at = row * ld + col;
  if (pairs) {
    mm_store_pairs(block, lane, a, b, rows, static_cast<uint16_t*>(to) + at, ld, cols - col);
  } else {
    mm_store_each(block, lane, a, rows, to, f32, at, ld, cols - col);
    mm_store_each(block, lane, b, rows, to, f32, at + 32, ld, cols - col - 32);
  }
}

// src(c0, c1, a, b): columns c0 .. c0 + 31 and c1 .. c1 + 31 of this lane's row of
// the tile, called by the whole warp.  row0: the warp's first row of the result.
template <int EPI, class Source>
__device__ __forceinline__ void mm_epilogue(const MmParams& p, int64_t row0, int64_t tile_n, int lane,
                                            uint32_t* block, Source src) {
  const int64_t row = row0 + lane;
  const int rows = mm_rows(p, row0);  // < 1: only src is called
  float a[32], b[32];
  if constexpr (EPI == MM_OUT) {
    const float scale = p.scale ? *p.scale : 1.0f;
    const MmOutRow to = mm_out_row(p, row0);
    for (int c = 0; c < p.tn; c += 64) {
      const int64_t col = tile_n * p.tn + c;
      src(c, c + 32, a, b);
      if (col >= p.N) continue;
      if (!p.accum_in && !p.accum_out && !p.base) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          a[j] *= scale;
          b[j] *= scale;
        }
        mm_store_64(block, lane, a, b, rows, to.out, p.out_f32, p.out_pairs, to.row, to.ld, col, p.N);
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 32; ++j) block[lane * kMmPitch + j] = __float_as_uint(h ? b[j] : a[j]);
        const int64_t at = col + 32 * h + lane;
        mm_by_rows(
            block, lane, rows, at < p.N,
            [&](int r, uint32_t w) {
              float x = __uint_as_float(w);
              if (p.accum_in) x += p.accum_in[(row0 + r) * p.accum_ld + at];
              if (!p.accum_out) x *= scale;
              if (p.base) x += mm_load(p.base, p.out_f32, (to.row + r) * p.base_ld + at);
              return x;
            },
            [&](int r, float x) {
              if (p.accum_out)
                p.accum_out[(row0 + r) * p.accum_ld + at] = x;
              else
                mm_store(to.out, p.out_f32, (to.row + r) * to.ld + at, x);
            });
      }
    }
  } else if constexpr (EPI == MM_LSE) {
    // exponentials to base 2 of z log2(e), relative to a row's largest so far
    int64_t t = -1;
    if (lane < rows) t = mm_token(p.targets, p.idx64, row);
    const int64_t hit = t >= 0 && t < p.V ? t - p.token0 - tile_n * p.tn : -1;
    float m = -INFINITY, s = 0.0f;
    for (int c = 0; c < p.tn; c += 64) {
      src(c, c + 32, a, b);
      const int64_t left = p.N - tile_n * p.tn - c;
      if (hit >= c && hit < c + 64) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (hit == c + j) p.picked[row] = a[j];
          if (hit == c + 32 + j) p.picked[row] = b[j];
        }
      }
      if (left < 64) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j >= left) a[j] = -INFINITY;
          if (j + 32 >= left) b[j] = -INFINITY;
        }
      }
      float top = fmaxf(a[0], b[0]);
#pragma unroll
      for (int j = 1; j < 32; ++j) top = fmaxf(top, fmaxf(a[j], b[j]));
      top *= kMmLog2e;
      if (top > m) {
        s *= mm_exp2(m - top);
        m = top;
      }
      const float ref = m == -INFINITY ? 0.0f : m;  // no difference of infinities
      float sa = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        sa += mm_exp2(fmaf(a[j], kMmLog2e, -ref));
        sb += mm_exp2(fmaf(b[j], kMmLog2e, -ref));
      }
      s += sa + sb;
    }
    if (lane < rows) p.part[tile_n * p.M + row] = make_float2(m, s);
  } else if constexpr (EPI == MM_ERROR) {
    int64_t hit = -1;
    float lse = 0.0f, w = 0.0f;  // of a masked row, whose logits are zeros
    if (lane < rows) {
      const int64_t t = mm_token(p.targets, p.idx64, row);
      if (t >= 0 && t < p.V) {
        hit = t - p.token0 - tile_n * p.tn;
        lse = p.lse[row];
        w = p.dloss[row * p.dloss_step] / *p.scale;
      }
    }
    for (int c = 0; c < p.tn; c += 64) {
      const int64_t col = tile_n * p.tn + c;
      src(c, c + 32, a, b);
      if (col >= p.N) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        a[j] = mm_exp(a[j] - lse);
        b[j] = mm_exp(b[j] - lse);
      }
      if (hit >= c && hit < c + 64) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (hit == c + j) a[j] -= 1.0f;
          if (hit == c + 32 + j) b[j] -= 1.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        a[j] *= w;
        b[j] *= w;
      }
      for (int k = 0; k < p.parts; ++k) {
        mm_store_pairs(block, lane, a, b, rows, static_cast<uint16_t*>(p.error) + k * p.error_plane + row0 * p.error_ld + col,
                       p.error_ld, p.N - col);
        if (k + 1 < p.parts) {  // what is left for the next part
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            a[j] -= Elem<__nv_bfloat16>::widen1(mm_narrow(a[j]));
            b[j] -= Elem<__nv_bfloat16>::widen1(mm_narrow(b[j]));
          }
        }
      }
    }
  } else {
    const int half = p.tn / 2;
    for (int c = 0; c < half; c += 64) {
      const int64_t col = tile_n * half + c;
      float d[32], e[32];
      src(c, half + c, a, b);
      src(c + 32, half + c + 32, d, e);
      if (col >= p.N) continue;
      if (p.gate) mm_store_64(block, lane, a, d, rows, p.gate, p.out_f32, p.out_pairs, row0, p.gate_ld, col, p.N);
      if (p.up) mm_store_64(block, lane, b, e, rows, p.up, p.out_f32, p.out_pairs, row0, p.up_ld, col, p.N);
      if (p.act == VCOLL_SILU) {
        mm_gate<VCOLL_SILU>(a, b);
        mm_gate<VCOLL_SILU>(d, e);
      } else if (p.act == VCOLL_GELU) {
        mm_gate<VCOLL_GELU>(a, b);
        mm_gate<VCOLL_GELU>(d, e);
      } else {
        mm_gate<VCOLL_GELU_TANH>(a, b);
        mm_gate<VCOLL_GELU_TANH>(d, e);
      }
      mm_store_64(block, lane, a, d, rows, p.out, p.out_f32, p.out_pairs, row0, p.out_ld, col, p.N);
    }
  }
}

}  // namespace vcoll
