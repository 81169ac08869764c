// Layer norm and its gradient for rows that a team of up to 16 warps holds in
// registers (instantiated for fp32 and bf16 in norm_f32.cu and norm_bf16.cu).
//
// Both are bound by memory: each reads its rows once and writes once.  A team
// of p.warps warps takes a row, R chunks of 32 * E columns a warp
// (row_access.cuh); CTAs stay resident and their teams walk the rows with the
// grid's stride.  The rows ahead are on their way meanwhile: each thread
// fetches its own pieces into a ring of slots in shared memory
// (cp.async), which costs no registers and needs no barrier; the team meets at
// one barrier a row, where its warps exchange their partial sums.
//
// Forward: a warp takes the mean and the squared deviations of its own
// columns, and the team joins them: with n_w, m_w, q_w a warp's number of
// columns, mean and squares, mean = sum(n_w m_w) / D and the squares are
// sum(q_w + n_w (m_w - mean)^2), which cancels no more than the two-pass form
// does.  Backward: the sums over g and g h of a row need one exchange; the
// sums over the rows for the weight and the bias stay in the registers of the
// thread that owns the column, and a CTA leaves one row of each in the
// workspace (vc_norm_wsum adds these up).
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
};

// The first column of a thread's chunk r.
template <typename T, int A>
__device__ __forceinline__ int team_col(const Team& t, int r) {
  return (t.warp + t.warps * r) * 32 * kLane<T> + t.lane * A;
}

}  // namespace

// The ring starts as zeros: columns past a row's end are never fetched and
// stay so.
__device__ __forceinline__ void clear_ring(char* smem, int bytes) {
  for (int k = threadIdx.x * 16; k < bytes; k += blockDim.x * 16)
    *reinterpret_cast<uint4*>(smem + k) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// Shared memory: the ring [stage][r][thread] of 16 bytes and the teams'
// partial sums.  Weight and bias are read for each row, from L1.
template <typename T, int A, int R, bool KEEP>
__global__ void __launch_bounds__(512, R >= 4 ? 1 : 2) vc_norm_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Pieces<T, A>;
  constexpr int E = P::E, S = norm_stages(R, false);
  extern __shared__ __align__(16) char smem[];
  const int threads = blockDim.x, D = (int)p.D;
  const Team t(p.warps);
  char* ring = smem + threadIdx.x * 16;
  const int slot = threads * 16;  // from one slot of a thread to its next
  float2* red = reinterpret_cast<float2*>(smem + S * R * slot) + t.index * 2 * t.warps;

  const int64_t teams = (int64_t)gridDim.x * (threads / 32 / p.warps);
  const int64_t first = (int64_t)blockIdx.x * (threads / 32 / p.warps) + t.index;
  auto fetch = [&](int64_t i, int s) {
    if (i < p.N)
#pragma unroll
      for (int r = 0; r < R; ++r)
        P::fetch(ring + (s * R + r) * slot, elem_at<T>(p.x, i * p.x_ld), team_col<T, A>(t, r), D);
    fetch_commit();
  };
  clear_ring(smem, S * R * slot);
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(first + s * teams, s);
  // columns of a warp
  auto columns = [&](int warp) {
    int n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) n += min(max(D - (warp + t.warps * r) * 32 * E, 0), 32 * E);
    return n;
  };
  const bool full = columns(t.warp) == R * 32 * E;
  const float cols = (float)max(columns(t.warp), 1), cols_of = (float)columns(t.lane);
  int s = 0, parity = 0;
  for (int64_t i = first; i < p.N; i += teams) {
    fetch_wait<S - 1>();
    float f[R][E], sx = 0.0f, sy = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Elem<T>::widen(*reinterpret_cast<const uint4*>(ring + (s * R + r) * slot), f[r]);
#pragma unroll
      for (int e = 0; e < E; e += 2) add2(sx, sy, sx, sy, f[r][e], f[r][e + 1]);
    }
    const float sum = warp_sum(sx + sy);
    fetch(i + S * teams, s);  // the slot has been read
    s = s + 1 == S ? 0 : s + 1;
    const float local = sum / cols;
    if (!full)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (team_col<T, A>(t, r) + P::offset(e) >= D) f[r][e] = local;
    float qx = 0.0f, qy = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float dx, dy;
        add2(dx, dy, f[r][e], f[r][e + 1], -local, -local);
        fma2(qx, qy, dx, dy, dx, dy, qx, qy);
      }
    float sq = warp_sum(qx + qy), mean = local;
    if (t.warps > 1) {
      float2* now = red + parity * t.warps;
      parity ^= 1;
      if (t.lane == 0) now[t.warp] = make_float2(sum, sq);
      t.meet();
      const float2 o = t.lane < t.warps ? now[t.lane] : make_float2(0.0f, 0.0f);
      mean = warp_sum(o.x) / (float)D;
      const float d = t.lane < t.warps && cols_of > 0.0f ? o.x / cols_of - mean : 0.0f;
      sq = warp_sum(fmaf(cols_of * d, d, o.y));
    }
    const float rstd = rsqrtf(sq / (float)D + p.eps);
    char* y = elem_at<T>(p.y, i * p.y_ld);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = team_col<T, A>(t, r);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        add2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], -mean, -mean);
        mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], rstd, rstd);
      }
      if constexpr (KEEP) {
        if (!full)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (c + P::offset(e) >= D) f[r][e] = 0.0f;
        keep8<T, A>(f[r], c, (t.warp + t.warps * r) * (32 * E / kBlock8), D, p.codes + i * p.codes_ld,
                    p.scales + i * ((D + kBlock8 - 1) / kBlock8));
      }
      float w[E], b[E];
      P::weights(p.weight, p.wbf16, c, D, 1.0f, w);
      P::weights(p.bias, p.wbf16, c, D, 0.0f, b);
#pragma unroll
      for (int e = 0; e < E; e += 2)
        fma2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], w[e], w[e + 1], b[e], b[e + 1]);
      P::store(y, c, D, f[r]);
    }
    if (t.warp == 0 && t.lane == 0) {
      if (p.mean) p.mean[i] = mean;
      if (p.rstd) p.rstd[i] = rstd;
    }
  }
}

// Shared memory: the ring [stage] of gradient and x [r][thread] of 16 bytes
// each (KEPT: instead of x the codes [r][warp] of 32 * E bytes, in the order of
// the columns, and the scales [r][thread] of 2 fp32), the row's statistics
// [thread] of 2 fp32; and the teams' partial sums.
template <typename T, int A, int R, bool KEPT>
__global__ void __launch_bounds__(512, 1) vc_norm_grad_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Pieces<T, A>;
  constexpr int E = P::E, S = norm_stages(R, true);
  // scales that a thread's pieces of a chunk need: their blocks of 128 columns
  constexpr int SC = 32 * E / kBlock8 == 2 && A < E ? 2 : 1;
  extern __shared__ __align__(16) char smem[];
  const int threads = blockDim.x, tid = threadIdx.x, D = (int)p.D;
  const int blocks = (D + kBlock8 - 1) / kBlock8;
  const Team t(p.warps);
  const int stage = norm_grad_slot_bytes(R, E, KEPT) * threads;
  char* gslot = smem + tid * 16;
  char* xslot = smem + R * threads * 16 + tid * (KEPT ? E : 16);
  char* cslot = smem + R * threads * (16 + E) + tid * 8;  // KEPT: scales
  char* sslot = smem + stage - threads * 8 + tid * 8;
  float2* red = reinterpret_cast<float2*>(smem + S * stage) + t.index * 2 * t.warps;

  const int64_t teams = (int64_t)gridDim.x * (threads / 32 / p.warps);
  const int64_t first = (int64_t)blockIdx.x * (threads / 32 / p.warps) + t.index;
  auto fetch = [&](int64_t i, int s) {
    if (i < p.N) {
      const int at = s * stage;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int c = team_col<T, A>(t, r);
        P::fetch(gslot + at + r * threads * 16, elem_at<T>(p.grad, i * p.grad_ld), c, D);
        if constexpr (KEPT) {
          // a warp's codes as they lie: pieces of E bytes whatever A is (rows of
          // codes are 16-byte aligned and padded)
          const int lin = c + t.lane * (E - A);
          if (lin < D) fetch_async<E>(xslot + at + r * threads * E, p.codes + i * p.codes_ld + lin);
#pragma unroll
          for (int k = 0; k < SC; ++k)
            if (c + k * kBlock8 < D)
              fetch_async<4>(cslot + at + r * threads * 8 + k * 4,
                             p.scales + i * blocks + c / kBlock8 + k);
        } else {
          P::fetch(xslot + at + r * threads * 16, elem_at<T>(p.x, i * p.x_ld), c, D);
        }
      }
      if constexpr (!KEPT) fetch_async<4>(sslot + at, p.mean + i);
      fetch_async<4>(sslot + at + 4, p.rstd + i);
    }
    fetch_commit();
  };
  clear_ring(smem, S * stage);
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(first + s * teams, s);
  float dw[R][E], db[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[r][e] = db[r][e] = 0.0f;

  int s = 0, parity = 0;
  for (int64_t i = first; i < p.N; i += teams) {
    fetch_wait<S - 1>();
    if constexpr (KEPT && A < E) __syncwarp();  // codes that other lanes fetched
    const int at = s * stage;
    const float2 stat = *reinterpret_cast<const float2*>(sslot + at);
    const float rstd = stat.y;
    // columns past the row's end have a gradient of 0, so they add nothing
    float f[R][E], h[R][E], s1x = 0.0f, s1y = 0.0f, s2x = 0.0f, s2y = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Elem<T>::widen(*reinterpret_cast<const uint4*>(gslot + at + r * threads * 16), f[r]);
      if constexpr (KEPT) {
        const char* from = xslot + at + r * threads * E;
        const float2 scale = *reinterpret_cast<const float2*>(cslot + at + r * threads * 8);
        uint32_t word[2] = {0u, 0u};
        if constexpr (A < E) {
          from -= t.lane * (E - A);  // this lane's first column
#pragma unroll
          for (int e = 0; e < E; ++e)
            word[e / 4] |= (uint32_t)(uint8_t)from[P::offset(e)] << (8 * (e % 4));
        } else if constexpr (E == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(from);
          word[0] = v.x;
          word[1] = v.y;
        } else {
          word[0] = *reinterpret_cast<const uint32_t*>(from);
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
          h[r][e] = code_value(word[e / 4], e % 4) * (SC == 2 && P::offset(e) >= kBlock8 ? scale.y : scale.x);
      } else {
        Elem<T>::widen(*reinterpret_cast<const uint4*>(xslot + at + r * threads * 16), h[r]);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          add2(h[r][e], h[r][e + 1], h[r][e], h[r][e + 1], -stat.x, -stat.x);
          mul2(h[r][e], h[r][e + 1], h[r][e], h[r][e + 1], rstd, rstd);
        }
      }
      float w[E];
      P::weights(p.weight, p.wbf16, team_col<T, A>(t, r), D, 1.0f, w);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        fma2(dw[r][e], dw[r][e + 1], f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], dw[r][e], dw[r][e + 1]);
        add2(db[r][e], db[r][e + 1], db[r][e], db[r][e + 1], f[r][e], f[r][e + 1]);
        mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], w[e], w[e + 1]);  // g from here on
        add2(s1x, s1y, s1x, s1y, f[r][e], f[r][e + 1]);
        fma2(s2x, s2y, f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], s2x, s2y);
      }
    }
    float s1 = warp_sum(s1x + s1y), s2 = warp_sum(s2x + s2y);
    fetch(i + S * teams, s);  // the slot has been read
    s = s + 1 == S ? 0 : s + 1;
    if (!p.y) continue;
    if (t.warps > 1) {
      float2* now = red + parity * t.warps;
      parity ^= 1;
      if (t.lane == 0) now[t.warp] = make_float2(s1, s2);
      t.meet();
      const float2 o = t.lane < t.warps ? now[t.lane] : make_float2(0.0f, 0.0f);
      s1 = warp_sum(o.x);
      s2 = warp_sum(o.y);
    }
    s1 /= -(float)D;
    s2 /= -(float)D;
    char* dx = elem_at<T>(p.y, i * p.y_ld);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        add2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], s1, s1);
        fma2(f[r][e], f[r][e + 1], h[r][e], h[r][e + 1], s2, s2, f[r][e], f[r][e + 1]);
        mul2(f[r][e], f[r][e + 1], f[r][e], f[r][e + 1], rstd, rstd);
      }
      P::store(dx, team_col<T, A>(t, r), D, f[r]);
    }
  }
  if (!p.part) return;
  // the CTA's sums: its teams add theirs up in the ring's memory, in order
  fetch_wait<0>();
  const int count = threads / 32 / p.warps;
  float* rows = reinterpret_cast<float*>(smem);  // [2][E * R][team's thread]
  const int width = p.warps * 32, own = t.warp * 32 + t.lane;
  for (int k = 0; k < count; ++k) {
    __syncthreads();
    if (t.index != k) continue;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float* a = rows + (r * E + e) * width + own;
        float* b = a + R * E * width;
        if (k) {
          dw[r][e] = *a + dw[r][e];
          db[r][e] = *b + db[r][e];
        }
        if (k + 1 < count) {
          *a = dw[r][e];
          *b = db[r][e];
        } else {
          const int c = team_col<T, A>(t, r) + P::offset(e);
          if (c < D) {
            p.part[(size_t)blockIdx.x * 2 * D + c] = dw[r][e];
            p.part[(size_t)(blockIdx.x * 2 + 1) * D + c] = db[r][e];
          }
        }
      }
  }
}

}  // namespace vcoll
