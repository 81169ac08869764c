// Device helpers of the layer norm and 8-bit activation kernels.
#pragma once

#include "device_common.cuh"
#include "layers_internal.h"
#include "row_access.cuh"

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
__device__ __forceinline__ float load_weight(const void* w, int bf16, int64_t i, float none) {
  if (!w) return none;
  return bf16 ? load1<__nv_bfloat16>(w, i) : load1<float>(w, i);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// A thread's pieces of one chunk of a row, A elements each; c: its first column.
template <typename T, int A>
struct Pieces {
  static constexpr int E = kLane<T>, BYTES = A * Elem<T>::kBytes;
  // element e of the thread's E is column c + offset(e)
  static __device__ __forceinline__ constexpr int offset(int e) { return e / A * 32 * A + e % A; }

  static __device__ __forceinline__ void fetch(void* slot, const void* row, int c, int D) {
#pragma unroll
    for (int j = 0; j < E / A; ++j)
      if (c + j * 32 * A < D)
        fetch_async<BYTES>(static_cast<char*>(slot) + j * BYTES, elem_at<T>(row, c + j * 32 * A));
  }
  // The weight (or bias) of the thread's columns, in either type, from a place
  // that allows accesses of A elements; ones or zeros where there is none.
  static __device__ __forceinline__ void weights(const void* w, int bf16, int c, int D, float none,
                                                 float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / A; ++j) {
      float g[A];
#pragma unroll
      for (int a = 0; a < A; ++a) g[a] = none;
      const int at = c + j * 32 * A;
      if (w && at < D) {
        if (bf16) {
          Raw<__nv_bfloat16, A> v;
          v.load(elem_at<__nv_bfloat16>(w, at));
          v.widen(g);
        } else {
          Raw<float, A> v;
          v.load(elem_at<float>(w, at));
          v.widen(g);
        }
      }
#pragma unroll
      for (int a = 0; a < A; ++a) f[j * A + a] = g[a];
    }
  }
  static __device__ __forceinline__ void load(Raw<T, A> (&v)[E / A], const void* row, int64_t c, int64_t D) {
#pragma unroll
    for (int j = 0; j < E / A; ++j) {
      if (c + j * 32 * A < D) v[j].load_stream(elem_at<T>(row, c + j * 32 * A));
      else v[j].zero();
    }
  }
  static __device__ __forceinline__ void widen(const Raw<T, A> (&v)[E / A], float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / A; ++j) {
      float g[A];
      v[j].widen(g);
#pragma unroll
      for (int a = 0; a < A; ++a) f[j * A + a] = g[a];
    }
  }
  static __device__ __forceinline__ void store(void* row, int64_t c, int64_t D, const float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E / A; ++j) {
      if (c + j * 32 * A >= D) break;
      float g[A];
#pragma unroll
      for (int a = 0; a < A; ++a) g[a] = f[j * A + a];
      Raw<T, A> o;
      o.narrow(g);
      o.store_stream(elem_at<T>(row, c + j * 32 * A));
    }
  }
};

// ------------------------------------------------------- 8-bit activations
// A block's largest magnitude is taken on the bits without the sign: as whole
// numbers they order the finite values, the infinity above them and every NaN
// above that.
struct Scale8 {
  float scale, unit;
  uint32_t mask;  // of the codes: 0 where all of them are 0
};
__device__ __forceinline__ Scale8 scale8(uint32_t top_bits) {
  Scale8 s;
  const float top = __uint_as_float(top_bits);
  const bool finite = top_bits < 0x7F800000u, some = finite && top >= kTiny8;
  s.scale = some ? __fdiv_rn(top, 127.0f) : finite ? 0.0f : __uint_as_float(0x7FC00000u);
  s.unit = some ? __fdiv_rn(127.0f, top) : 0.0f;
  s.mask = some ? 0xFFFFFFFFu : 0u;
  return s;
}
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The product rounded to the nearest integer, ties to even, in the low byte:
// the sum with 1.5 * 2^23 is rounded to a whole number, whose two's complement
// ends the sum's bits (|product| <= 127.5).  An add where a conversion
// instruction would have an eighth of its rate.
__device__ __forceinline__ uint32_t code_bits(float x, float unit) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, unit), 12582912.0f));
}
// code k of a word as fp32: the byte plus 128 as the end of 2^23's bits, less
// 2^23 + 128; both steps exact.
__device__ __forceinline__ float code_value(uint32_t word, int k) {
  const uint32_t up = word ^ 0x80808080u;
  return __uint_as_float(__byte_perm(up, 0x4B000000u, 0x7540 | k)) - 8388736.0f;
}

// Keeps a lane's E values of a chunk: its codes and, from one lane, the
// chunk's scales.  Values past the row's end are 0.  c: the lane's first
// column; block: the chunk's first block.
template <typename T, int A>
__device__ __forceinline__ void keep8(const float (&f)[kLane<T>], int64_t c, int64_t block, int64_t D,
                                      int8_t* codes, float* scales) {
  constexpr int E = kLane<T>, B = 32 * E / kBlock8;  // blocks of a chunk
  const int lane = threadIdx.x & 31;
  // offset of element e from the lane's first column, and its block
  auto offset = [](int e) { return Pieces<T, A>::offset(e); };
  auto block_of = [&](int e) { return B == 1 ? 0 : A == E ? lane >> 4 : offset(e) / kBlock8; };
  uint32_t top[B];
#pragma unroll
  for (int b = 0; b < B; ++b) top[b] = 0u;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t m = magnitude_bits(f[e]);
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (block_of(e) == b) top[b] = max(top[b], m);
  }
  Scale8 s[B];
#pragma unroll
  for (int b = 0; b < B; ++b) s[b] = scale8(__reduce_max_sync(~0u, top[b]));
  uint32_t word[E / 4];
#pragma unroll
  for (int k = 0; k < E; k += 4) {
    uint32_t q[4], mask = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int in = block_of(k + e);
      const float unit = B == 1 || in == 0 ? s[0].unit : s[B - 1].unit;
      mask = B == 1 || in == 0 ? s[0].mask : s[B - 1].mask;
      q[e] = code_bits(f[k + e], unit);
    }
    word[k / 4] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410) & mask;
  }
  const int64_t end = (D + 15) & ~(int64_t)15;
#pragma unroll
  for (int j = 0; j < E / A; ++j) {
    const int64_t at = c + j * 32 * A;
    if (at >= end) break;
    if constexpr (A == 8) *reinterpret_cast<uint2*>(codes + at) = make_uint2(word[0], word[1]);
    else if constexpr (A == 4) *reinterpret_cast<uint32_t*>(codes + at) = word[j];
    else if constexpr (A == 2)
      *reinterpret_cast<uint16_t*>(codes + at) = (uint16_t)(word[j / 2] >> (16 * (j % 2)));
    else codes[at] = (int8_t)(word[j / 4] >> (8 * (j % 4)));
  }
  const int64_t blocks = (D + kBlock8 - 1) / kBlock8;
  if (lane == 0 && block < blocks) scales[block] = s[0].scale;
  if (B == 2 && lane == 16 && block + 1 < blocks) scales[block + 1] = s[B - 1].scale;
}

}  // namespace

}  // namespace vcoll
