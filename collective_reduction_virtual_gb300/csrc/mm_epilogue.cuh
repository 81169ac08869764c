// What becomes of a tile of a product (MmEpilogue), a warp for 32 of its rows.
//
// The accumulators arrive as the tensor cores leave them: a lane holds a row,
// 32 columns at a time.  What goes along a row (its maximum and sum, what its
// target decides) is done there, in registers.  What is stored goes through a 32
// x 33 block of shared memory, after which a lane holds two adjacent columns of
// every second row: a warp's stores are 64 or 128 adjacent bytes of two rows.
// The loops are kept short rather than unrolled: a tile's first pass through
// them waits for instructions (4000 of them took longer than a small product).
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
// e^x: off by 2 ulp and by |x| 2^-23, since x log2(e) is rounded (and log2(e) itself).
// Where |x| is large the value is small beside those it is added to: of a softmax's
// sum, whose largest term is 1; of 1 + e^-g; of a density.
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
// act = g * s, act' = s + g * ds, with what mm_low and mm_finite make of an infinite g.
// The exact gelu takes erfcf where g < 0, since 1 + erf loses the bits of a small
// result.  Where a factor has come to 0 or 1, ds is 0 whatever g * g is.
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
    const float both = s * (1.0f - s);
    ds = both == 0.0f ? 0.0f : both * c * (1.0f + 0.134145f * g * g);
  }
}
// The limits at infinity: act(-inf) = -0, act'(inf) = 1, act'(-inf) = 0, where the
// factor 0 must not meet an infinite g.  A NaN stays one.
constexpr float kMmHighest = 3.402823466e38f;
__device__ __forceinline__ float mm_low(float g) { return g < -kMmHighest ? -kMmHighest : g; }
__device__ __forceinline__ float mm_finite(float g) { return g > kMmHighest ? kMmHighest : mm_low(g); }

// Where a row of the result goes.
struct MmOutRow {
  void* out;
  int64_t ld, row;  // within out
};
__device__ __forceinline__ MmOutRow mm_out_row(const MmParams& p, int64_t row) {
  const bool second = p.M1 && row >= p.M1;
  return {second ? p.out2 : p.out, second ? p.out2_ld : p.out_ld, second ? row - p.M1 : row};
}
// of a warp's rows from row0 on: those that are the result's
__device__ __forceinline__ int mm_rows(const MmParams& p, int64_t row0) {
  const int64_t end = !p.M1 ? p.M : row0 >= p.M1 ? p.M1 + p.M2 : p.M2;
  return (int)(end - row0 < p.warp_rows ? end - row0 : p.warp_rows);
}

// A warp's block of 32 rows and 32 columns of the result, as its lanes take it: two
// adjacent columns in every second row where two can be moved at once (WIDE), else a
// column of every row, so that a warp's access is one piece of two rows or of one.
template <bool WIDE>
struct MmBlock {
  int rows;       // of the result in it
  int64_t col;    // this lane's first column
  int64_t left;   // columns from there on that are the result's
  int row, at;    // this lane's first row, and its place in the block
  static constexpr int STEP = WIDE ? 2 : 1, COUNT = WIDE ? 16 : 32;

  __device__ __forceinline__ MmBlock(int rows_, int64_t col0, int64_t cols, int lane) : rows(rows_) {
    const int c = WIDE ? (lane & 15) * 2 : lane;
    row = WIDE ? lane >> 4 : 0;
    at = row * kMmPitch + c;
    col = col0 + c;
    left = cols - col;
  }
};

// x = (in + first * x) * then.  in may be NULL.
struct MmAdd {
  const void* in;
  int64_t in_at, in_ld;
  void* out;
  int64_t out_at, out_ld;
  float first, then;
};
// What is added to a block.  All loads are issued at once, from places within the
// matrix whatever the row and column, and without a condition between them, which
// they would wait for: a load waits longer than all else takes.
template <bool IN32, bool WIDE>
__device__ __forceinline__ void mm_add_load(const MmAdd& h, const MmBlock<WIDE>& b, float (&x)[32]) {
  using Block = MmBlock<WIDE>;
  if (!h.in || b.rows <= 0 || !__any_sync(~0u, b.left > 0)) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    return;
  }
  const int64_t col = b.left > 0 ? b.col : b.col + b.left - Block::STEP;  // the last there are
#pragma unroll
  for (int i = 0; i < Block::COUNT; ++i) {
    const int r = b.row + i * Block::STEP < b.rows ? b.row + i * Block::STEP : b.rows - 1;
    const int64_t at = h.in_at + r * h.in_ld + col;
    if (WIDE && IN32) {
      const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(h.in) + at);
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    } else if (WIDE) {
      x[2 * i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(h.in) + at));
    } else if (IN32) {
      x[i] = static_cast<const float*>(h.in)[at];
    } else {
      x[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(h.in)[at] << 16);
    }
  }
  if (WIDE && !IN32) {
#pragma unroll
    for (int i = 0; i < Block::COUNT; ++i)
      Elem<__nv_bfloat16>::widen2(__float_as_uint(x[2 * i]), x[2 * i], x[2 * i + 1]);
  }
}
template <bool OUT32, bool WIDE>
__device__ __forceinline__ void mm_add_store(const MmAdd& h, const MmBlock<WIDE>& b, const float (&x)[32],
                                             const float* block) {
  using Block = MmBlock<WIDE>;
  if (b.left <= 0) return;
#pragma unroll
  for (int i = 0; i < Block::COUNT; ++i) {
    const int r = i * Block::STEP;
    if (b.row + r >= b.rows) break;
    const float* from = block + b.at + r * kMmPitch;
    const int64_t at = h.out_at + (b.row + r) * h.out_ld + b.col;
    if (WIDE) {
      const float y = (x[2 * i] + h.first * from[0]) * h.then, z = (x[2 * i + 1] + h.first * from[1]) * h.then;
      if (OUT32)
        *reinterpret_cast<float2*>(static_cast<float*>(h.out) + at) = make_float2(y, z);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(h.out) + at) = mm_narrow2(y, z);
    } else {
      mm_store(h.out, OUT32, at, (x[i] + h.first * from[0]) * h.then);
    }
  }
}
// A block of fp32, or of bf16 whose rows do not allow 4-byte accesses.
template <bool WIDE>
__device__ __forceinline__ void mm_store_block(const MmBlock<WIDE>& b, const float* block, float scale, void* out, int f32,
                                               int64_t at, int64_t ld) {
  if (b.left <= 0) return;
#pragma unroll 4
  for (int r = b.row; r < b.rows; r += MmBlock<WIDE>::STEP) {
    const float* from = block + b.at + (r - b.row) * kMmPitch;
    const int64_t to = at + r * ld + b.col;
    if (WIDE)
      *reinterpret_cast<float2*>(static_cast<float*>(out) + to) = make_float2(from[0] * scale, from[1] * scale);
    else
      mm_store(out, f32, to, from[0] * scale);
  }
}

// What an epilogue will add, fetched to L2 a unit ahead: a lane a row of the warp's
// 32.
__device__ __forceinline__ void mm_prefetch_added(const MmParams& p, int64_t row0, int64_t tile_n, int c0, int c1, int lane) {
  if (!p.accum_in && !p.base) return;
  const int rows = mm_rows(p, row0);
  const int64_t col = tile_n * p.tn + c0, end = p.N < tile_n * p.tn + c1 ? p.N : tile_n * p.tn + c1;
  if (lane >= rows || col >= end) return;
  const int es = p.accum_in || p.out_f32 ? 4 : 2;
  const int64_t at = p.accum_in ? (row0 + lane) * p.accum_ld : (mm_out_row(p, row0).row + lane) * p.base_ld;
  const char* first = static_cast<const char*>(p.accum_in ? (const void*)p.accum_in : p.base) + (at + col) * es;
  const char* last = first + (end - col) * es - 1;
  for (uintptr_t line = (uintptr_t)first & ~(uintptr_t)127; line <= (uintptr_t)last; line += 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
}

__device__ __forceinline__ void mm_to_block(float* block, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) block[lane * kMmPitch + j] = v[j];
  __syncwarp();
}

template <bool IN32, bool OUT32, bool WIDE, class Source>
__device__ __forceinline__ void mm_add_blocks(const MmAdd& h, int rows, int64_t col0, int64_t cols, int c0, int c1,
                                              int lane, float* block, Source src) {
  for (int c = c0; c < c1; c += 32) {
    const MmBlock<WIDE> b(rows, col0 + c, cols, lane);
    float x[32];
    src(c, x);
    mm_to_block(block, lane, x);
    mm_add_load<IN32>(h, b, x);
    mm_add_store<OUT32>(h, b, x, block);
    __syncwarp();
  }
}

// 64 columns as bf16, two to a word: a warp's stores are 128 adjacent bytes of a
// row (with 64 bytes of two rows the block's training batch took 4 % longer).
__device__ __forceinline__ void mm_store_64(float* block, int lane, const float (&a)[32], const float (&b)[32],
                                            int rows, uint16_t* to, int64_t ld, int64_t left) {
  uint32_t* words = reinterpret_cast<uint32_t*>(block);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    words[lane * kMmPitch + j] = mm_narrow2(a[2 * j], a[2 * j + 1]);
    words[lane * kMmPitch + 16 + j] = mm_narrow2(b[2 * j], b[2 * j + 1]);
  }
  __syncwarp();
  to += 2 * lane;
  if (2 * lane + 1 < left) {
#pragma unroll 8
    for (int r = 0; r < rows; ++r, to += ld) *reinterpret_cast<uint32_t*>(to) = words[r * kMmPitch + lane];
  } else if (2 * lane < left) {
    for (int r = 0; r < rows; ++r, to += ld) *to = (uint16_t)words[r * kMmPitch + lane];
  }
  __syncwarp();
}

template <int ACT>
__device__ __forceinline__ void mm_gate(float (&g)[32], const float (&u)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float s, ds;
    mm_act(ACT, g[j], s, ds);
    g[j] = mm_low(g[j]) * (s * u[j]);
  }
}

// What a row's exponentials are relative to: its largest logit so far, or where that is
// infinite zero, since infinities have no difference.  A logit of +infinity then makes
// the sum infinite, and with it lse.
__device__ __forceinline__ float mm_ref(float top) { return fabsf(top) == INFINITY ? 0.0f : top; }

// What a lane's row brings besides its sums, loaded before they are waited for.
struct MmRow {
  float scale;  // MM_OUT
  int64_t hit;  // the tile's column of the row's target, or one that it has not
  float lse, w;  // of a masked row, whose logits are zeros: 0
};
template <int EPI>
__device__ __forceinline__ MmRow mm_row(const MmParams& p, int64_t row0, int64_t tile_n, int lane) {
  MmRow r = {1.0f, -1, 0.0f, 0.0f};
  if constexpr (EPI == MM_OUT) {
    if (p.scale) r.scale = *p.scale;
  } else if constexpr (EPI == MM_LSE || EPI == MM_ERROR) {
    if (lane < mm_rows(p, row0)) {
      const int64_t t = mm_token(p.targets, p.idx64, row0 + lane);
      const bool inside = t >= 0 && t < p.V;
      if (inside) r.hit = t - p.token0 - tile_n * p.tn;
      if (EPI == MM_ERROR) {
        const float lse = p.lse[row0 + lane], w = p.dloss[(row0 + lane) * p.dloss_step] / *p.scale;
        r.lse = inside ? lse : 0.0f;
        r.w = inside ? w : 0.0f;
      }
    }
  }
  return r;
}

// src(c, v): columns c .. c + 31 of this lane's row of the tile, called by the
// whole warp; columns c0 .. c1 - 1 are this warp's.  row0: its first row of the
// result.
template <int EPI, class Source>
__device__ __forceinline__ void mm_epilogue(const MmParams& p, int64_t row0, int64_t tile_n, int c0, int c1,
                                            const MmRow& mine, int lane, float* block, Source src) {
  const int64_t row = row0 + lane;
  const int rows = mm_rows(p, row0);  // < 1: only src is called
  float v[32];
  if constexpr (EPI == MM_OUT) {
    const float scale = mine.scale;
    const MmOutRow to = mm_out_row(p, row0);
    const bool add = p.accum_in || p.accum_out || p.base;
    if (!add && !p.out_f32 && p.out_pairs) {
      float w[32];
      for (int c = c0; c < c1; c += 64) {
        const int64_t col = tile_n * p.tn + c;
        src(c, v);
        src(c + 32, w);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          v[j] *= scale;
          w[j] *= scale;
        }
        mm_store_64(block, lane, v, w, rows, static_cast<uint16_t*>(to.out) + to.row * to.ld + col, to.ld, p.N - col);
      }
      return;
    }
    if (add) {
      const MmAdd how = {p.accum_in ? (const void*)p.accum_in : p.base,
                         p.accum_in ? row0 * p.accum_ld : to.row * p.base_ld, p.accum_in ? p.accum_ld : p.base_ld,
                         p.accum_out ? (void*)p.accum_out : to.out,
                         p.accum_out ? row0 * p.accum_ld : to.row * to.ld, p.accum_out ? p.accum_ld : to.ld,
                         p.base || p.accum_scaled ? scale : 1.0f,
                         p.base || p.accum_scaled || p.accum_out ? 1.0f : scale};
      const bool out32 = p.accum_out || p.out_f32, in32 = p.accum_in || out32;
      // pairs of columns do not reach past the last one
      const bool wide = p.N % 2 == 0 && (p.accum_in || !p.base || p.out_pairs) && (p.accum_out || p.out_pairs);
      const int64_t col0 = tile_n * p.tn;
      if (in32 && out32 && wide)
        mm_add_blocks<true, true, true>(how, rows, col0, p.N, c0, c1, lane, block, src);
      else if (in32 && out32)
        mm_add_blocks<true, true, false>(how, rows, col0, p.N, c0, c1, lane, block, src);
      else if (in32)
        mm_add_blocks<true, false, false>(how, rows, col0, p.N, c0, c1, lane, block, src);
      else if (wide)
        mm_add_blocks<false, false, true>(how, rows, col0, p.N, c0, c1, lane, block, src);
      else
        mm_add_blocks<false, false, false>(how, rows, col0, p.N, c0, c1, lane, block, src);
      return;
    }
    for (int c = c0; c < c1; c += 32) {
      src(c, v);
      mm_to_block(block, lane, v);
      if (p.out_f32 && p.out_pairs && p.N % 2 == 0)
        mm_store_block(MmBlock<true>(rows, tile_n * p.tn + c, p.N, lane), block, scale, to.out, 1, to.row * to.ld, to.ld);
      else
        mm_store_block(MmBlock<false>(rows, tile_n * p.tn + c, p.N, lane), block, scale, to.out, p.out_f32,
                       to.row * to.ld, to.ld);
      __syncwarp();
    }
  } else if constexpr (EPI == MM_LSE) {
    // exponentials relative to a row's largest logit so far, which is kept as it is: its
    // own exponential is exactly 1, and it meets a rounding only in the sum that is lse
    const int64_t hit = mine.hit;
    float m = -INFINITY, s = 0.0f;
    for (int c = c0; c < c1; c += 32) {
      src(c, v);
      const int64_t left = p.N - tile_n * p.tn - c;
      if (hit >= c && hit < c + 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (hit == c + j) p.picked[row] = v[j];
      }
      if (left < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= left) v[j] = -INFINITY;
      }
      float top = v[0];
#pragma unroll
      for (int j = 1; j < 32; ++j) top = fmaxf(top, v[j]);
      if (top > m) {
        s *= mm_exp(m - top);
        m = top;
      }
      const float ref = mm_ref(m);
      float part[4] = {};
#pragma unroll
      for (int j = 0; j < 32; ++j) part[j % 4] += mm_exp(v[j] - ref);
      s += (part[0] + part[1]) + (part[2] + part[3]);
    }
    if (lane < rows && c0 < c1) p.part[(tile_n * (p.tn / (c1 - c0)) + (c0 ? 1 : 0)) * p.M + row] = make_float2(m, s);
  } else if constexpr (EPI == MM_ERROR) {
    // e, the one matrix that has to exist: of bf16 operands in one bf16, half a step of 2^-8
    // off, as a program holds it that keeps its logits' gradient (results of bf16 are then off
    // by 1.14 to 1.16 times their own rounding; two parts would double both products' work);
    // of fp32 operands in three, which hold its 24 bits
    const int64_t hit = mine.hit;
    const float lse = mine.lse, w = mine.w;
    float x[32];
    for (int c = c0; c < c1; c += 64) {
      const int64_t col = tile_n * p.tn + c;
      src(c, v);
      src(c + 32, x);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] = mm_exp(v[j] - lse);
        x[j] = mm_exp(x[j] - lse);
      }
      if (hit >= c && hit < c + 64) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (hit == c + j) v[j] -= 1.0f;
          if (hit == c + 32 + j) x[j] -= 1.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] *= w;
        x[j] *= w;
      }
      for (int k = 0; k < p.parts; ++k) {  // a part, and what it leaves for the next
        mm_store_64(block, lane, v, x, rows,
                    static_cast<uint16_t*>(p.error) + k * p.error_plane + row0 * p.error_ld + col, p.error_ld,
                    p.N - col);
        if (k + 1 < p.parts) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[j] -= Elem<__nv_bfloat16>::widen1(mm_narrow(v[j]));
            x[j] -= Elem<__nv_bfloat16>::widen1(mm_narrow(x[j]));
          }
        }
      }
    }
  } else if (!p.out_f32 && p.out_pairs && p.act != VCOLL_GELU) {
    const int half = p.tn / 2;
    float w[32], u[32];
    for (int c = c0 / 2; c < c1 / 2; c += 64) {
      const int64_t col = tile_n * half + c, left = p.N - col;
      for (int k = 0; k < 2; ++k) {  // tensor memory is read again rather than held
        uint16_t* to = static_cast<uint16_t*>(k ? p.up : p.gate);
        const int64_t ld = k ? p.up_ld : p.gate_ld;
        if (!to) continue;
        src(k * half + c, v);
        src(k * half + c + 32, w);
        mm_store_64(block, lane, v, w, rows, to + row0 * ld + col, ld, left);
      }
      src(c, v);
      src(half + c, u);
      if (p.act == VCOLL_SILU) mm_gate<VCOLL_SILU>(v, u);
      else mm_gate<VCOLL_GELU_TANH>(v, u);
      src(c + 32, w);
      src(half + c + 32, u);
      if (p.act == VCOLL_SILU) mm_gate<VCOLL_SILU>(w, u);
      else mm_gate<VCOLL_GELU_TANH>(w, u);
      mm_store_64(block, lane, v, w, rows, static_cast<uint16_t*>(p.out) + row0 * p.out_ld + col, p.out_ld, left);
    }
  } else {
    // (the exact gelu's code is too long to be repeated for 64 columns)
    // 16 columns of gate and the same of up beside each other; a lane takes one of
    // them in every second row
    const int half = p.tn / 2, at = lane & 15;
    for (int c = c0 / 2; c < c1 / 2; c += 16) {
      const int64_t col = tile_n * half + c + at;
      src(c, half + c, v);
      mm_to_block(block, lane, v);
      if (col < p.N) {
#pragma unroll 4
        for (int r = lane >> 4; r < rows; r += 2) {
          const float g = block[r * kMmPitch + at], u = block[r * kMmPitch + at + 16];
          float s, ds;
          mm_act(p.act, g, s, ds);
          if (p.gate) mm_store(p.gate, p.out_f32, (row0 + r) * p.gate_ld + col, g);
          if (p.up) mm_store(p.up, p.out_f32, (row0 + r) * p.up_ld + col, u);
          mm_store(p.out, p.out_f32, (row0 + r) * p.out_ld + col, mm_low(g) * (s * u));
        }
      }
      __syncwarp();
    }
  }
}

}  // namespace vcoll
