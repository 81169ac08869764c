// How the layer kernels walk a row: a warp takes chunks of 32 * E columns, E
// per lane, E elements making 16 bytes of the input type.  A lane's columns
// are E / A groups of A adjacent ones, one access each, and the lanes' groups
// lie side by side, so that every access of a warp is one contiguous piece.
// A == E (16-byte accesses) needs addresses, row strides and widths that are
// multiples of E; A == 2 and A == 1 take rows of any even, and any, width.
#pragma once

#include "device_common.cuh"

namespace vcoll {

template <typename T>
constexpr int kLane = 16 / Elem<T>::kBytes;  // E

// The raw bits of A elements, A * sizeof(T) bytes up to 16 (a group of 8 fp32
// is two of them, used for outputs beside bf16 inputs).
template <typename T, int A>
struct Raw {
  static constexpr int kBytes = A * Elem<T>::kBytes;
  static_assert(kBytes == 2 || kBytes == 4 || kBytes == 8 || kBytes == 16 || kBytes == 32, "");
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0;
  }
  // read once: evict first
  __device__ __forceinline__ void load_stream(const void* p) {
    if constexpr (kBytes == 2) {
      asm volatile("ld.global.cs.u16 %0, [%1];" : "=r"(w[0]) : "l"(p));  // zeros above
    } else if constexpr (kBytes == 4) {
      asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else if constexpr (kBytes == 8) {
      asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4)
        asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[k]), "=r"(w[k + 1]), "=r"(w[k + 2]), "=r"(w[k + 3])
                     : "l"((const char*)p + 4 * k));
    }
  }
  // read again soon by this or another CTA
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kBytes == 2) {
      w[0] = *static_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *static_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *static_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const uint4 v = static_cast<const uint4*>(p)[k / 4];
        w[k] = v.x;
        w[k + 1] = v.y;
        w[k + 2] = v.z;
        w[k + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store_stream(void* p) const {
    if constexpr (kBytes == 2) {
      __stcs(static_cast<uint16_t*>(p), (uint16_t)w[0]);
    } else if constexpr (kBytes == 4) {
      __stcs(static_cast<uint32_t*>(p), w[0]);
    } else if constexpr (kBytes == 8) {
      __stcs(static_cast<uint2*>(p), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4)
        __stcs(static_cast<uint4*>(p) + k / 4, make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]));
    }
  }
  __device__ __forceinline__ void widen(float (&f)[A]) const {
    if constexpr (Elem<T>::kBytes == 4) {
#pragma unroll
      for (int a = 0; a < A; ++a) f[a] = __uint_as_float(w[a]);
    } else if constexpr (A == 1) {
      f[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int a = 0; a < A; a += 2) Elem<__nv_bfloat16>::widen2(w[a / 2], f[a], f[a + 1]);
    }
  }
  // Puts the bits in their place among the words of 16 bytes, first: the first
  // element's number there (words are zero so far where A * kBytes == 2).
  __device__ __forceinline__ void into(uint32_t (&word)[4], int first) const {
    if constexpr (kBytes == 2) {
      word[first / 2] |= w[0] << (16 * (first % 2));
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) word[first * Elem<T>::kBytes / 4 + k] = w[k];
    }
  }
  // computed values: a NaN becomes the canonical one
  __device__ __forceinline__ void narrow(const float (&f)[A]) {
    if constexpr (Elem<T>::kBytes == 4) {
#pragma unroll
      for (int a = 0; a < A; ++a) w[a] = __float_as_uint(f[a]);
    } else if constexpr (A == 1) {
      const __nv_bfloat16 h = __float2bfloat16_rn(f[0]);
      w[0] = *reinterpret_cast<const uint16_t*>(&h);
    } else {
#pragma unroll
      for (int a = 0; a < A; a += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[a], f[a + 1]);
        w[a / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ const char* elem_at(const void* base, int64_t i) {
  return static_cast<const char*>(base) + i * Elem<T>::kBytes;
}
template <typename T>
__device__ __forceinline__ char* elem_at(void* base, int64_t i) {
  return static_cast<char*>(base) + i * Elem<T>::kBytes;
}

// Which piece of which row a warp takes, where a row has `pieces` of them.
struct RowPiece {
  int64_t row, piece;
  __device__ __forceinline__ RowPiece(int64_t unit, int64_t pieces) {
    if ((unit | pieces) >> 32) {
      row = unit / pieces;
    } else {  // a quarter of the instructions
      row = (uint32_t)unit / (uint32_t)pieces;
    }
    piece = unit - row * pieces;
  }
};

__device__ __forceinline__ int64_t token_at(const void* tokens, int idx64, int64_t i) {
  return idx64 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// Two fp32 operations in one instruction, each rounded as the single ones are.
__device__ __forceinline__ void add2(float& x, float& y, float ax, float ay, float bx, float by) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void mul2(float& x, float& y, float ax, float ay, float bx, float by) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void fma2(float& x, float& y, float ax, float ay, float bx, float by,
                                     float cx, float cy) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by), "f"(cx), "f"(cy));
}

// cp.async: each thread fetches its own pieces into its own slots of shared
// memory and waits for them alone, so a ring of such slots keeps several rows
// in flight without registers and without a barrier between threads.
template <int BYTES>
__device__ __forceinline__ void fetch_async(void* slot, const void* from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
  else if constexpr (BYTES == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
  else {  // below the smallest asynchronous copy
    static_assert(BYTES == 2, "");
    *static_cast<uint16_t*>(slot) = *static_cast<const uint16_t*>(from);
  }
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace vcoll
