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

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

// The columns of a lane in a warp's group of R chunks of 32 * E adjacent
// columns.  In what follows c is the lane's first column in the row of D
// columns; FULL: the warp's whole group lies inside the row.
template <typename T, int A, int R>
struct Lanes {
  static constexpr int E = kLane<T>, BYTES = A * Elem<T>::kBytes;
  static constexpr int kColumns = R * 32 * E;
  static __device__ __forceinline__ int first(int lane) { return lane * A; }
  // column of element e of chunk r, from the first one
  static __device__ __forceinline__ constexpr int offset(int r, int e) {
    return r * 32 * E + e / A * 32 * A + e % A;
  }
  template <bool FULL>
  static __device__ __forceinline__ bool inside(int r, int e, int c, int D) {
    return FULL || c + offset(r, e) < D;
  }
  // slots: one of 16 bytes for each r, `step` bytes apart
  template <bool FULL>
  static __device__ __forceinline__ void fetch(char* slots, int step, const char* row, int c, int D) {
    const char* from = row + (int64_t)c * Elem<T>::kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += A)
        if (inside<FULL>(r, e, c, D))
          fetch_async<BYTES>(slots + r * step + e * Elem<T>::kBytes, from + offset(r, e) * Elem<T>::kBytes);
  }
  template <bool FULL>
  static __device__ __forceinline__ void load(uint4 (&raw)[R], const char* row, int c, int D) {
    const char* from = row + (int64_t)c * Elem<T>::kBytes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < E; e += A) {
        Raw<T, A> v;
        if (inside<FULL>(r, e, c, D)) v.load_stream(from + offset(r, e) * Elem<T>::kBytes);
        else v.zero();
        v.into(word, e);
      }
      raw[r] = make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
  template <bool FULL>
  static __device__ __forceinline__ void store(char* row, int c, int D, const float (&f)[R][E]) {
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
        if (inside<FULL>(r, e, c, D)) o.store_stream(to + offset(r, e) * Elem<T>::kBytes);
      }
  }
  // The weight (or bias), of type TW, of chunk r's columns, from a place that
  // allows accesses of A elements.
  template <typename TW, bool FULL>
  static __device__ __forceinline__ void weights(const void* w, int r, int c, int D, float (&f)[E]) {
    const char* from = elem_at<TW>(w, c);
#pragma unroll
    for (int e = 0; e < E; e += A) {
      float g[A];
      Raw<TW, A> v;
      if (inside<FULL>(r, e, c, D)) v.load(from + offset(r, e) * Elem<TW>::kBytes);
      else v.zero();
      v.widen(g);
#pragma unroll
      for (int a = 0; a < A; ++a) f[e + a] = g[a];
    }
  }
  template <typename TW, bool FULL>
  static __device__ __forceinline__ void scale_by(const void* w, int c, int D, float (&f)[R][E]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[E];
      weights<TW, FULL>(w, r, c, D, v);
#pragma unroll
      for (int e = 0; e < E; e += 2) mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], v[e], v[e + 1]);
    }
  }
  template <typename TW, bool FULL>
  static __device__ __forceinline__ void affine_by(const void* w, const void* b, int c, int D,
                                                   float (&f)[R][E]) {
    if (w && b) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float v[E], u[E];
        weights<TW, FULL>(w, r, c, D, v);
        weights<TW, FULL>(b, r, c, D, u);
#pragma unroll
        for (int e = 0; e < E; e += 2)
          fma2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], v[e], v[e + 1], u[e], u[e + 1]);
      }
    } else if (w) {
      scale_by<TW, FULL>(w, c, D, f);
    } else if (b) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float u[E];
        weights<TW, FULL>(b, r, c, D, u);
#pragma unroll
        for (int e = 0; e < E; e += 2) add2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], u[e], u[e + 1]);
      }
    }
  }
  // f * weight + bias, each of which may be absent
  template <bool FULL>
  static __device__ __forceinline__ void affine(const void* w, const void* b, int bf16, int c, int D,
                                                float (&f)[R][E]) {
    if (bf16) affine_by<__nv_bfloat16, FULL>(w, b, c, D, f);
    else affine_by<float, FULL>(w, b, c, D, f);
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
// Codes k and k + 1 of a word times a scale: a byte plus 128 as the end of
// 2^23's bits, less 2^23 + 128 (both steps exact), times the scale.
__device__ __forceinline__ void code_values(uint32_t word, int k, float scale, float& x, float& y) {
  const uint32_t up = word ^ 0x80808080u;
  add2(x, y, __uint_as_float(__byte_perm(up, 0x4B000000u, 0x7540 | k)),
       __uint_as_float(__byte_perm(up, 0x4B000000u, 0x7540 | (k + 1))), -8388736.0f, -8388736.0f);
  mul2(x, y, x, y, scale, scale);
}

// The four codes of 4 values.
__device__ __forceinline__ uint32_t code_word(const float* f, const Scale8& s) {
  return __byte_perm(__byte_perm(code_bits(f[0], s.unit), code_bits(f[1], s.unit), 0x0040),
                     __byte_perm(code_bits(f[2], s.unit), code_bits(f[3], s.unit), 0x0040), 0x5410) &
         s.mask;
}

// The largest of R values over each LB adjacent lanes.  Halves of the values
// change hands first, so that R values take little more shuffles than one: the
// lane ends with the one of value group_of(lane).
template <int R, int LB>
struct GroupTop {
  static constexpr int kEach = LB / R;  // adjacent lanes that end with the same value
  static __device__ __forceinline__ int group_of(int lane) { return lane / kEach % R; }
  static __device__ __forceinline__ uint32_t top(uint32_t (&v)[R]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = LB / 2, n = R; d; d >>= 1) {
      if (n > 1) {
        n /= 2;
#pragma unroll
        for (int k = 0; k < R / 2; ++k)
          if (k < n) {
            const uint32_t mine = lane & d ? v[k + n] : v[k], other = lane & d ? v[k] : v[k + n];
            v[k] = max(mine, __shfl_xor_sync(~0u, other, d));
          }
      } else {
        v[0] = max(v[0], __shfl_xor_sync(~0u, v[0], d));
      }
    }
    return v[0];
  }
};

// Keeps a warp's group of values: the codes and the scales of its blocks.
// Values past the row's end are 0.  col: the group's first column, a multiple
// of 128; c = col + Lanes::first(lane).
template <typename T, int A, int R>
__device__ __forceinline__ void keep8(const float (&f)[R][kLane<T>], int col, int c, int D, int8_t* codes,
                                      float* scales) {
  using P = Lanes<T, A, R>;
  constexpr int E = P::E;
  const int lane = threadIdx.x & 31, end = (D + 15) & ~15;
  if constexpr (A == E) {
    // a block is LB adjacent lanes' access: each lane computes the scale of one
    // of its R blocks
    constexpr int LB = kBlock8 / E;
    using G = GroupTop<R, LB>;
    uint32_t top[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      top[r] = 0u;
#pragma unroll
      for (int e = 0; e < E; ++e) top[r] = max(top[r], magnitude_bits(f[r][e]));
    }
    const Scale8 mine = scale8(G::top(top));
    const int first = lane & ~(LB - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Scale8 s;
      s.unit = __shfl_sync(~0u, mine.unit, first + r * G::kEach);
      s.mask = s.unit != 0.0f ? 0xFFFFFFFFu : 0u;
      if (c + P::offset(r, 0) >= end) continue;
      int8_t* at = codes + c + P::offset(r, 0);
      if constexpr (E == 8)
        *reinterpret_cast<uint2*>(at) = make_uint2(code_word(f[r], s), code_word(f[r] + 4, s));
      else *reinterpret_cast<uint32_t*>(at) = code_word(f[r], s);
    }
    const int at = col + G::group_of(lane) * 32 * E + first * E;  // the block's first column
    if (lane % G::kEach == 0 && at < D) scales[at / kBlock8] = mine.scale;
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

// ------------------------------------------------------------ narrow rows
// A row of up to G * E columns is taken by G lanes (8, 16 or 32), accesses of A
// elements side by side, so that a warp takes 32 / G rows at a time.
template <typename T, int A, int G>
struct Group {
  static constexpr int E = kLane<T>, BYTES = Elem<T>::kBytes;
  int sub, c;  // which of the warp's rows, first column
  __device__ __forceinline__ Group() {
    const int lane = threadIdx.x & 31;
    sub = lane / G;
    c = lane % G * A;
  }
  static __device__ __forceinline__ constexpr int offset(int e) { return e / A * G * A + e % A; }

  __device__ __forceinline__ uint4 load(const char* row, int D, bool in) const {
    uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < E; e += A) {
      Raw<T, A> v;
      if (in && c + offset(e) < D) v.load_stream(row + (c + offset(e)) * BYTES);
      else v.zero();
      v.into(word, e);
    }
    return make_uint4(word[0], word[1], word[2], word[3]);
  }
  __device__ __forceinline__ void store(char* row, int D, const float (&f)[E]) const {
#pragma unroll
    for (int e = 0; e < E; e += A) {
      float g[A];
#pragma unroll
      for (int a = 0; a < A; ++a) g[a] = f[e + a];
      Raw<T, A> o;
      o.narrow(g);
      if (c + offset(e) < D) o.store_stream(row + (c + offset(e)) * BYTES);
    }
  }
  __device__ __forceinline__ void weights(const void* w, int bf16, int D, float none, float (&f)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e)
      f[e] = c + offset(e) < D ? load_weight(w, bf16, c + offset(e), none) : 0.0f;
  }
  static __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int d = G / 2; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
  }
  // Which of a row's two blocks of 128 columns element e lies in.
  __device__ __forceinline__ int block_of(int e) const {
    return G * E <= kBlock8 ? 0 : (c + offset(e)) / kBlock8;
  }
  // Keeps the row's values (0 past its end): codes and scales.  Every lane of
  // the warp calls it; `in`: the row exists.
  __device__ __forceinline__ void keep(const float (&f)[E], int D, bool in, int8_t* codes,
                                       float* scales) const {
    // whole accesses of a row of two blocks: half of its lanes have each
    constexpr bool HALVES = G * E > kBlock8 && A == E;
    constexpr int B = G * E <= kBlock8 || HALVES ? 1 : 2, L = HALVES ? G / 2 : G;
    uint32_t top[B];
#pragma unroll
    for (int b = 0; b < B; ++b) top[b] = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (B == 1 || block_of(e) == b) top[b] = max(top[b], magnitude_bits(f[e]));
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int d = L / 2; d; d >>= 1) top[b] = max(top[b], __shfl_xor_sync(~0u, top[b], d));
    Scale8 s[B];
#pragma unroll
    for (int b = 0; b < B; ++b) s[b] = scale8(top[b]);
    if (!in) return;
    const int end = (D + 15) & ~15;
    uint32_t word[E / 4];
#pragma unroll
    for (int k = 0; k < E; k += 4)  // four elements lie in one block
      word[k / 4] = code_word(f + k, s[B == 2 && block_of(k) == 1 ? B - 1 : 0]);
#pragma unroll
    for (int e = 0; e < E; e += A) {
      const int at = c + offset(e);
      if (at >= end) break;
      if constexpr (A == 8) *reinterpret_cast<uint2*>(codes + at) = make_uint2(word[0], word[E / 4 - 1]);
      else if constexpr (A == 4) *reinterpret_cast<uint32_t*>(codes + at) = word[e / 4];
      else if constexpr (A == 2)
        *reinterpret_cast<uint16_t*>(codes + at) = (uint16_t)(word[e / 4] >> (8 * (e % 4)));
      else codes[at] = (int8_t)(word[e / 4] >> (8 * (e % 4)));
    }
    // rows of fewer than G * E columns may have no second block
    if (c == 0)
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (b * kBlock8 < D) scales[b] = s[b].scale;
    if (HALVES && c == kBlock8 && c < D) scales[1] = s[0].scale;
  }
  // h from codes and scales
  __device__ __forceinline__ void kept(const int8_t* codes, const float* scales, int D, bool in,
                                       float (&h)[E]) const {
    uint32_t word[2] = {0u, 0u};
    float scale[E / 4];
#pragma unroll
    for (int e = 0; e < E; e += A) {
      const int at = c + offset(e);
      const bool has = in && at < D;
      if (e % 4 == 0) scale[e / 4] = has ? scales[at / kBlock8] : 0.0f;
      if (!has) continue;
      if constexpr (A == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(codes + at));
        word[0] = v.x;
        word[1] = v.y;
        scale[E / 4 - 1] = scale[0];
      } else if constexpr (A == 4) {
        word[e / 4] = __ldcs(reinterpret_cast<const uint32_t*>(codes + at));
      } else {
#pragma unroll
        for (int a = 0; a < A; ++a)
          word[(e + a) / 4] |= (uint32_t)(uint8_t)codes[at + a] << (8 * ((e + a) % 4));
      }
    }
    if constexpr (A == 8) scale[E / 4 - 1] = scale[0];
#pragma unroll
    for (int e = 0; e < E; e += 2) code_values(word[e / 4], e % 4, scale[e / 4], h[e], h[e + 1]);
  }
};

}  // namespace

}  // namespace vcoll
