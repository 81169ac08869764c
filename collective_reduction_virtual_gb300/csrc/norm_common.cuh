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

// The columns of a lane in a warp's group of R chunks (R * 32 * E columns).
// Plainly, chunk r is 32 * E adjacent columns.  With BLOCKS, and whole accesses
// (A == E), each block of 128 columns belongs to LANES lanes, all R accesses of
// a lane lying in one block: its scale is then computed, or fetched, once for
// R * E values, and an access of the warp is pieces of LANES * 16 bytes.
template <typename T, int A, int R, bool BLOCKS>
struct Lanes {
  static constexpr int E = kLane<T>, BYTES = A * Elem<T>::kBytes;
  static constexpr int kColumns = R * 32 * E;
  static constexpr bool kBlocks = BLOCKS && A == E;
  static constexpr int LANES = 128 / (R * E) < 32 ? 128 / (R * E) : 32;
  // first column of lane in the group, and column of element e of access r from there
  static __device__ __forceinline__ int first(int lane) {
    return kBlocks ? lane / LANES * kBlock8 + lane % LANES * E : lane * A;
  }
  static __device__ __forceinline__ constexpr int offset(int r, int e) {
    return kBlocks ? r * LANES * E + e : r * 32 * E + e / A * 32 * A + e % A;
  }

  // In what follows c is the lane's first column in the row of D columns;
  // full: the warp's whole group lies inside the row.
  static __device__ __forceinline__ bool inside(int r, int e, int c, int D, bool full) {
    return full || c + offset(r, e) < D;
  }
  // slots: one of 16 bytes for each r, `step` bytes apart
  static __device__ __forceinline__ void fetch(char* slots, int step, const char* row, int c, int D,
                                               bool full) {
    const char* from = row + (int64_t)c * Elem<T>::kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += A)
        if (inside(r, e, c, D, full))
          fetch_async<BYTES>(slots + r * step + e * Elem<T>::kBytes, from + offset(r, e) * Elem<T>::kBytes);
  }
  static __device__ __forceinline__ void load(uint4 (&raw)[R], const char* row, int c, int D, bool full) {
    const char* from = row + (int64_t)c * Elem<T>::kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < E; e += A) {
        Raw<T, A> v;
        if (inside(r, e, c, D, full)) v.load_stream(from + offset(r, e) * Elem<T>::kBytes);
        else v.zero();
        v.into(word, e);
      }
      raw[r] = make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
  static __device__ __forceinline__ void store(char* row, int c, int D, bool full, const float (&f)[R][E]) {
    char* to = row + (int64_t)c * Elem<T>::kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += A) {
        float g[A];
#pragma unroll
        for (int a = 0; a < A; ++a) g[a] = f[r][e + a];
        Raw<T, A> o;
        o.narrow(g);
        if (inside(r, e, c, D, full)) o.store_stream(to + offset(r, e) * Elem<T>::kBytes);
      }
  }
  // The weight (or bias) of access r's columns, in either type, from a place
  // that allows accesses of A elements; `none` where there is none.
  static __device__ __forceinline__ void weights(const void* w, int bf16, int r, int c, int D, bool full,
                                                 float none, float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = none;
    if (!w) return;
    if (bf16) {
      const char* from = elem_at<__nv_bfloat16>(w, c);
#pragma unroll
      for (int e = 0; e < E; e += A)
        if (inside(r, e, c, D, full)) {
          float g[A];
          Raw<__nv_bfloat16, A> v;
          v.load(from + offset(r, e) * 2);
          v.widen(g);
#pragma unroll
          for (int a = 0; a < A; ++a) f[e + a] = g[a];
        }
    } else {
      const char* from = elem_at<float>(w, c);
#pragma unroll
      for (int e = 0; e < E; e += A)
        if (inside(r, e, c, D, full)) {
          float g[A];
          Raw<float, A> v;
          v.load(from + offset(r, e) * 4);
          v.widen(g);
#pragma unroll
          for (int a = 0; a < A; ++a) f[e + a] = g[a];
        }
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

// The four codes of 4 values.
__device__ __forceinline__ uint32_t code_word(const float* f, const Scale8& s) {
  return __byte_perm(__byte_perm(code_bits(f[0], s.unit), code_bits(f[1], s.unit), 0x0040),
                     __byte_perm(code_bits(f[2], s.unit), code_bits(f[3], s.unit), 0x0040), 0x5410) &
         s.mask;
}

// Keeps a warp's group of values: the codes and the scales of its blocks.
// Values past the row's end are 0.  col: the group's first column, a multiple
// of 128; c = col + Lanes::first(lane).
template <typename T, int A, int R>
__device__ __forceinline__ void keep8(const float (&f)[R][kLane<T>], int col, int c, int D, int8_t* codes,
                                      float* scales) {
  using P = Lanes<T, A, R, true>;
  constexpr int E = P::E;
  const int lane = threadIdx.x & 31, end = (D + 15) & ~15;
  if constexpr (P::kBlocks) {
    uint32_t top = 0u;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, magnitude_bits(f[r][e]));
    if constexpr (P::LANES == 32) {
      top = __reduce_max_sync(~0u, top);
    } else {
#pragma unroll
      for (int d = P::LANES / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    }
    const Scale8 s = scale8(top);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (c + P::offset(r, 0) >= end) break;
      int8_t* at = codes + c + P::offset(r, 0);
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(at) = make_uint2(code_word(f[r], s), code_word(f[r] + 4, s));
      else *reinterpret_cast<uint32_t*>(at) = code_word(f[r], s);
    }
    if (lane % P::LANES == 0 && c < D) scales[c / kBlock8] = s.scale;
  } else {
    constexpr int B = 32 * E / kBlock8;  // blocks of a chunk, 4 elements of a lane in each
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int first = col + r * 32 * E + b * kBlock8;
        if (first >= D) break;
        const float* v = f[r] + 4 * b;
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, magnitude_bits(v[e]));
        const Scale8 s = scale8(__reduce_max_sync(~0u, top));
        const uint32_t word = code_word(v, s);
#pragma unroll
        for (int e = 0; e < 4; e += A) {
          const int at = c + P::offset(r, 4 * b + e);
          if (at >= end) break;
          if constexpr (A == 2) *reinterpret_cast<uint16_t*>(codes + at) = (uint16_t)(word >> (8 * e));
          else codes[at] = (int8_t)(word >> (8 * e));
        }
        if (lane == 0) scales[first / kBlock8] = s.scale;
      }
  }
}

}  // namespace

}  // namespace vcoll
