// Layer norm and its gradient for rows that a team of up to 16 warps holds in
// registers (instantiated for fp32 and bf16 in norm_f32.cu and norm_bf16.cu).
//
// Both are bound by memory: each reads its rows once and writes once.  A team
// of p.warps warps takes a row, R * 32 * E adjacent columns a warp (Lanes);
// CTAs stay resident and their teams walk the rows with the grid's stride.  The
// rows ahead are on their way meanwhile: each thread fetches its own pieces
// into a ring of slots in shared memory (cp.async), which costs no registers
// and needs no barrier.  A value is widened once and stays in a register until
// its result is stored; pairs of values share an instruction (f32x2), without
// which the issue of instructions would bound the kernels.
//
// Forward: the mean, then the squares of the deviations, then the outputs, in
// registers; the team's warps exchange their sums at two barriers.  Backward:
// the row's sums over g and g h need one; the sums over the rows for the
// weight and the bias stay in the registers of the thread that owns the
// column (of wide rows in shared memory), and a CTA leaves one row of each in
// the workspace (vc_norm_wsum adds these up).
//
// Measured: 32768 x 8192 bf16 forward 177 us, 6.1 TB/s, of which the measured
// copy does 6.7; 32768 x 4096 bf16 backward 131 us and 5 for vc_norm_wsum, 6.1
// TB/s.  With the 8-bit form, 16384 x 4096 bf16, 62 and 74 us (5.4 and 4.6
// TB/s), issue at 57 and 51 %.  Two CTAs of 256 threads are on an SM, held by 128
// registers; at 80 both spill.  Rows of 8 chunks a warp spill at 128, most of all
// the fp32 gradient from 8 bits above 8192 columns (300 bytes a thread: 10007 x
// 12288 314 us, 274 without the 8 bits).  Rows of single bf16 elements are copied
// to the ring synchronously and wait for it: 100003 x 1001 192 us forward and 430
// backward, three to five times what their bytes take.
#pragma once

#include "layers_internal.h"
#include "norm_common.cuh"
#include "row_access.cuh"

namespace vcoll {

namespace {

// The team of this thread: its number in the CTA, and its barrier.
struct Team {
  int warps, index, warp, lane;
  __device__ __forceinline__ explicit Team(int w) : warps(w) {
    lane = threadIdx.x & 31;
    index = (threadIdx.x >> 5) / w;
    warp = (threadIdx.x >> 5) - index * w;
  }
  __device__ __forceinline__ void meet() const {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
  }
  // Sums over the team of what each warp has summed, the same in every thread.
  // A place is written again after the team has met once more at the earliest:
  // callers alternate between two.
  __device__ __forceinline__ float sum(float v, float* place) const {
    if (lane == 0) place[warp] = v;
    meet();
    return warp_sum(lane < warps ? place[lane] : 0.0f);
  }
  __device__ __forceinline__ void sum2(float& a, float& b, float* place) const {
    float2* at = reinterpret_cast<float2*>(place);
    if (lane == 0) at[warp] = make_float2(a, b);
    meet();
    const float2 o = lane < warps ? at[lane] : make_float2(0.0f, 0.0f);
    a = warp_sum(o.x);
    b = warp_sum(o.y);
  }
};

// V adjacent sums, one store.
template <int V>
__device__ __forceinline__ void put_sums(float* to, const float* v) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
  else if constexpr (V == 2) *reinterpret_cast<float2*>(to) = make_float2(v[0], v[1]);
  else *to = *v;
}

// The ring starts as zeros: columns past a row's end are never fetched and
// stay so.
__device__ __forceinline__ void clear_ring(char* smem, int bytes) {
  for (int k = threadIdx.x * 16; k < bytes; k += blockDim.x * 16)
    *reinterpret_cast<uint4*>(smem + k) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

}  // namespace

// Shared memory: the ring [stage][r][thread] of 16 bytes and the teams'
// partial sums.  Weight and bias are read for each row, from L1.  MT: threads
// of a CTA at most.
template <typename T, int A, int R, int MT, bool KEEP>
__global__ void __launch_bounds__(MT, MT == 256 ? 2 : 1)
    vc_norm_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Lanes<T, A, R>;
  constexpr int E = P::E, S = norm_stages(R, E, false);
  extern __shared__ __align__(16) char smem[];
  const int threads = blockDim.x, D = (int)p.D;
  const Team t(p.warps);
  const int col = t.warp * P::kColumns, c = col + P::first(t.lane);
  char* ring = smem + threadIdx.x * 16;
  const int slot = threads * 16;  // from one slot of a thread to its next
  float* red = reinterpret_cast<float*>(smem + S * R * slot) + t.index * 4 * t.warps;

  const uint32_t rows = (uint32_t)p.N, teams = gridDim.x * (threads / 32 / p.warps);
  const uint32_t begin = blockIdx.x * (threads / 32 / p.warps) + t.index;
  clear_ring(smem, S * R * slot);
  // a warp whose columns all lie inside the row needs no guards
  auto work = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const char* x = elem_at<T>(p.x, begin * p.x_ld);
    char* y = elem_at<T>(p.y, begin * p.y_ld);
    const int64_t xstep = teams * p.x_ld * Elem<T>::kBytes, ystep = teams * p.y_ld * Elem<T>::kBytes;
    uint32_t ahead = begin;  // next row to fetch
    auto fetch = [&](int s) {
      if (ahead < rows) P::template fetch<FULL>(ring + s * R * slot, slot, x, c, D);
      fetch_commit();
      ahead += teams;
      x += xstep;
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(s);
    int s = 0;
    for (uint32_t i = begin; i < rows; i += teams, y += ystep) {
      fetch_wait<S - 1>();
      float f[R][E], sx = 0.0f, sy = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Elem<T>::widen(*reinterpret_cast<const uint4*>(ring + (s * R + r) * slot), f[r]);
#pragma unroll
        for (int e = 0; e < E; e += 2) add2(sx, sy, sx, sy, f[r][e], f[r][e + 1]);
      }
      float mean = warp_sum(sx + sy);
      fetch(s);  // the slot has been read
      s = s + 1 == S ? 0 : s + 1;
      if (t.warps > 1) mean = t.sum(mean, red);
      mean /= (float)D;
      float qx = 0.0f, qy = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          add2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], -mean, -mean);
          if (!P::template inside<FULL>(r, e, c, D)) f[r][e] = 0.0f;
          if (!P::template inside<FULL>(r, e + 1, c, D)) f[r][e + 1] = 0.0f;
          fma2(qx, qy, f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], qx, qy);
        }
      float var = warp_sum(qx + qy);
      if (t.warps > 1) var = t.sum(var, red + 2 * t.warps);
      const float rstd = rsqrtf(var / (float)D + p.eps);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; e += 2) mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], rstd, rstd);
      if constexpr (KEEP)
        keep8<T, A, R>(f, col, c, D, p.codes + i * p.codes_ld,
                       p.scales + (int64_t)i * ((D + kBlock8 - 1) / kBlock8));
      P::template affine<FULL>(p.weight, p.bias, p.wbf16, c, D, f);
      P::template store<FULL>(y, c, D, f);
      if (t.warp == 0 && t.lane == 0) {
        if (p.mean) p.mean[i] = mean;
        if (p.rstd) p.rstd[i] = rstd;
      }
    }
  };
  if (col + P::kColumns <= D) work(Bool<true>());
  else work(Bool<false>());
}

// Shared memory: the ring [stage] of gradient and x [r][thread] of 16 bytes
// each (KEPT: instead of x the codes, E bytes), and the teams' partial sums.
// Where A < E a warp's codes lie in the order of the columns.  The row's
// statistics and scales, which many lanes share, are loaded into registers one
// row ahead: as asynchronous copies to each lane's slot they would take more of
// the load/store unit's time than the rows themselves.
template <typename T, int A, int R, int MT, bool KEPT>
__global__ void __launch_bounds__(MT, MT == 256 ? 2 : 1)
    vc_norm_grad_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Lanes<T, A, R>;
  constexpr int E = P::E, S = norm_stages(R, E, true);
  // scales that a lane needs for a chunk: of its access's block, or of all
  constexpr int SC = A == E ? 1 : 32 * E / kBlock8;
  extern __shared__ __align__(16) char smem[];
  const int threads = blockDim.x, tid = threadIdx.x, D = (int)p.D;
  const int blocks = (D + kBlock8 - 1) / kBlock8;
  const Team t(p.warps);
  const int col = t.warp * P::kColumns, c = col + P::first(t.lane);
  const int stage = norm_grad_slot_bytes(R, E, KEPT) * threads;
  char* gslot = smem + tid * 16;
  char* xslot = smem + R * threads * 16 + tid * (KEPT ? E : 16);
  // the sums over the rows: in registers, or beside the ring, where they start
  // as zeros, too: [dw, db][r][k][thread] of 4 fp32 (fp32 rows leave room there
  // for the one alone)
  constexpr bool SUMS = norm_grad_smem_sums(R, E) > 0, BOTH = norm_grad_smem_sums(R, E) > 1;
  const int sums_bytes = norm_grad_smem_sums(R, E) * R * E * 4 * threads;
  float4* sums = reinterpret_cast<float4*>(smem + S * stage) + tid;
  float* red = reinterpret_cast<float*>(smem + S * stage + sums_bytes) + t.index * 4 * t.warps;

  const uint32_t rows = (uint32_t)p.N, teams = gridDim.x * (threads / 32 / p.warps);
  const uint32_t begin = blockIdx.x * (threads / 32 / p.warps) + t.index;
  float dw[R][E], db[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[r][e] = db[r][e] = 0.0f;
  clear_ring(smem, S * stage + sums_bytes);
  auto work = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const char* grad = elem_at<T>(p.grad, begin * p.grad_ld);
    const char* x = KEPT ? reinterpret_cast<const char*>(p.codes) + begin * p.codes_ld
                         : elem_at<T>(p.x, begin * p.x_ld);
    char* dx = p.y ? elem_at<T>(p.y, begin * p.y_ld) : nullptr;
    const int64_t gstep = teams * p.grad_ld * Elem<T>::kBytes;
    const int64_t xstep = KEPT ? teams * p.codes_ld : teams * p.x_ld * Elem<T>::kBytes;
    const int64_t dstep = p.y ? teams * p.y_ld * Elem<T>::kBytes : 0;
    uint32_t ahead = begin;  // next row to fetch
    auto fetch = [&](int s) {
      if (ahead < rows) {
        const int at = s * stage;
        P::template fetch<FULL>(gslot + at, threads * 16, grad, c, D);
        if constexpr (KEPT) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            // pieces of E bytes whatever A is: rows of codes are 16-byte aligned
            // and padded
            const int from = col + (r * 32 + t.lane) * E;
            if (FULL || from < D) {
              // beside rows of single bf16 elements, which are copied at once, the
              // codes are, too.  As asynchronous copies behind the others, four chunks
              // a warp, the last chunk's landed in the slot of the second or the third
              // (nvcc 13.0.88; other warps from run to run, with nothing else in
              // flight), though two copies of 4 bytes, or the codes first, landed where
              // they should: not a matter of the source's order
              if constexpr (P::BYTES < 4)
                *reinterpret_cast<uint2*>(xslot + at + r * threads * E) =
                    *reinterpret_cast<const uint2*>(x + from);
              else fetch_async<E>(xslot + at + r * threads * E, x + from);
            }
          }
        } else {
          P::template fetch<FULL>(xslot + at, threads * 16, x, c, D);
        }
      }
      fetch_commit();
      ahead += teams;
      grad += gstep;
      x += xstep;
    };
    float mean_next = 0.0f, rstd_next = 0.0f, scale_next[R][SC];
    auto look_ahead = [&](uint32_t row) {
      if (row >= rows) return;
      rstd_next = p.rstd[row];
      if constexpr (KEPT) {
        const float* scales = p.scales + (int64_t)row * blocks;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < SC; ++k) {
            const int at = c + r * 32 * E + k * kBlock8;
            scale_next[r][k] = FULL || at < D ? scales[at / kBlock8] : 0.0f;
          }
      } else {
        mean_next = p.mean[row];
      }
    };
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(s);
    look_ahead(begin);
    int s = 0, place = 0;
    for (uint32_t i = begin; i < rows; i += teams, dx += dstep) {
      fetch_wait<S - 1>();
      if constexpr (KEPT && A < E) __syncwarp();  // codes that other lanes fetched
      const int at = s * stage;
      [[maybe_unused]] const float mean = mean_next;
      const float rstd = rstd_next;
      float scale[R][SC];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < SC; ++k) scale[r][k] = KEPT ? scale_next[r][k] : 0.0f;
      look_ahead(i + teams);
      // columns past the row's end have a gradient of 0, so they add nothing
      float f[R][E], h[R][E];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Elem<T>::widen(*reinterpret_cast<const uint4*>(gslot + at + r * threads * 16), f[r]);
        if constexpr (KEPT) {
          const char* from = xslot + at + r * threads * E;
          uint32_t word[2] = {0u, 0u};
          if constexpr (A < E) {
            from -= t.lane * (E - A);  // this lane's first column
#pragma unroll
            for (int e = 0; e < E; ++e)
              word[e / 4] |= (uint32_t)(uint8_t)from[P::offset(0, e)] << (8 * (e % 4));
          } else if constexpr (E == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(from);
            word[0] = v.x;
            word[1] = v.y;
          } else {
            word[0] = *reinterpret_cast<const uint32_t*>(from);
          }
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float sc = scale[r][SC == 2 && e >= 4 ? 1 : 0];
            code_values(word[e / 4], e % 4, sc, h[r][e], h[r][e + 1]);
          }
        } else {
          Elem<T>::widen(*reinterpret_cast<const uint4*>(xslot + at + r * threads * 16), h[r]);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            add2(h[r][e], h[r][e + 1], h[r][e], h[r][e + 1], -mean, -mean);
            mul2(h[r][e], h[r][e + 1], h[r][e], h[r][e + 1], rstd, rstd);
          }
        }
        if constexpr (SUMS) {
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            float4* at = sums + (r * E + k) / 4 * threads;
            float4 w = *at;
            fma2(w.x, w.y, f[r][k], f[r][k + 1], h[r][k], h[r][k + 1], w.x, w.y);
            fma2(w.z, w.w, f[r][k + 2], f[r][k + 3], h[r][k + 2], h[r][k + 3], w.z, w.w);
            *at = w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2)
            fma2(dw[r][e], dw[r][e + 1], f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], dw[r][e], dw[r][e + 1]);
        }
        if constexpr (BOTH) {
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            float4* at = sums + (R * E + r * E + k) / 4 * threads;
            float4 b = *at;
            add2(b.x, b.y, b.x, b.y, f[r][k], f[r][k + 1]);
            add2(b.z, b.w, b.z, b.w, f[r][k + 2], f[r][k + 3]);
            *at = b;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) add2(db[r][e], db[r][e + 1], db[r][e], db[r][e + 1], f[r][e], f[r][e + 1]);
        }
      }
      if constexpr (!KEPT && !FULL) {
        // past the row's end h is -mean * rstd: where that is no finite number, 0
        // times it would reach the row's sum (one test a row: 8000 x 9001 fp32
        // 280 us, 366 with a selection for each value)
        if (!isfinite(mean * rstd)) {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (!P::template inside<FULL>(r, e, c, D)) h[r][e] = 0.0f;
        }
      }
      P::template affine<FULL>(p.weight, nullptr, p.wbf16, c, D, f);  // g
      float s1x = 0.0f, s1y = 0.0f, s2x = 0.0f, s2y = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          add2(s1x, s1y, s1x, s1y, f[r][e], f[r][e + 1]);
          fma2(s2x, s2y, f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], s2x, s2y);
        }
      float s1 = warp_sum(s1x + s1y), s2 = warp_sum(s2x + s2y);
      if constexpr (KEPT && A < E) __syncwarp();  // codes that other lanes have read
      fetch(s);  // the slot has been read
      s = s + 1 == S ? 0 : s + 1;
      if (!p.y) continue;
      if (t.warps > 1) {
        t.sum2(s1, s2, red + place);
        place ^= 2 * t.warps;
      }
      s1 /= -(float)D;
      s2 /= -(float)D;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          add2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], s1, s1);
          fma2(f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], s2, s2, f[r][e], f[r][e + 1]);
          mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], rstd, rstd);
        }
      P::template store<FULL>(dx, c, D, f);
    }
  };
  if (col + P::kColumns <= D) work(Bool<true>());
  else work(Bool<false>());
  if (!p.part) return;
  // rows of partial sums: stores of V adjacent columns (4096 x 4096 bf16: 24 us,
  // and 31 with single ones, of which a warp's lie 32 bytes apart)
  constexpr int V = A < 4 ? A : 4;
  float* part = p.part + (size_t)blockIdx.x * 2 * D;
  if constexpr (SUMS) {  // one team, each thread its own columns
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += V) {
        const int at = c + P::offset(r, e);
        const float* own = reinterpret_cast<const float*>(sums + (r * E + e) / 4 * threads) + e % 4;
        if (at < D) {
          put_sums<V>(part + at, own);
          put_sums<V>(part + D + at, BOTH ? own + R * E * threads : &db[r][e]);
        }
      }
    return;
  }
  // the CTA's sums: its teams add theirs up in the ring's memory, in order
  fetch_wait<0>();
  const int count = threads / 32 / p.warps;
  float* shared = reinterpret_cast<float*>(smem);  // [2][E * R][team's thread]
  const int width = p.warps * 32, own = t.warp * 32 + t.lane;
  for (int k = 0; k < count; ++k) {
    __syncthreads();
    if (t.index != k) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float* a = shared + (r * E + e) * width + own;
        float* b = a + R * E * width;
        if (k) {
          dw[r][e] = *a + dw[r][e];
          db[r][e] = *b + db[r][e];
        }
        if (k + 1 < count) {
          *a = dw[r][e];
          *b = db[r][e];
        }
      }
    if (k + 1 < count) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += V) {
        const int at = c + P::offset(r, e);
        if (at < D) {
          put_sums<V>(part + at, &dw[r][e]);
          put_sums<V>(part + D + at, &db[r][e]);
        }
      }
  }
}

}  // namespace vcoll
