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

// fp32 values of a thread's E elements lie 16 bytes apart per thread.
template <int E>
__device__ __forceinline__ void read_slots(const float* base, int threads, float (&f)[E]) {
#pragma unroll
  for (int k = 0; k < E; k += 4) {
    const float4 v = *reinterpret_cast<const float4*>(base + (size_t)(k / 4) * threads * 4);
    f[k] = v.x;
    f[k + 1] = v.y;
    f[k + 2] = v.z;
    f[k + 3] = v.w;
  }
}

// The weight (or bias) of a thread's columns of a chunk, past the end 0.
template <typename T, int A>
__device__ __forceinline__ void read_weight(const void* w, int bf16, int c, int D, float none,
                                            float (&f)[kLane<T>]) {
#pragma unroll
  for (int e = 0; e < kLane<T>; ++e) {
    const int at = c + Pieces<T, A>::offset(e);
    f[e] = at < D ? load_weight(w, bf16, at, none) : 0.0f;
  }
}

}  // namespace

// Shared memory: the ring [stage][r][thread] of 16 bytes, weight and bias
// [r][k][thread] of 4 fp32 (wide rows read them again each time: they would
// take the whole of it), and the teams' partial sums.
template <typename T, int A, int R, bool KEEP>
__global__ void __launch_bounds__(512, R == 8 ? 1 : 2) vc_norm_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Pieces<T, A>;
  constexpr int E = P::E, S = norm_stages(R, false);
  constexpr bool WS = norm_keeps_weight(R);
  extern __shared__ __align__(16) char smem[];
  const int threads = blockDim.x, tid = threadIdx.x, D = (int)p.D;
  const Team t(p.warps);
  char* ring = smem + tid * 16;
  const int slot = threads * 16;  // from one slot of a thread to its next
  float* weight = reinterpret_cast<float*>(smem + S * R * slot) + tid * 4;
  float* bias = weight + (size_t)R * E * threads;
  float2* red = reinterpret_cast<float2*>(smem + (S * R + (WS ? 2 * R * E / 4 : 0)) * slot) +
                t.index * 2 * t.warps;

  const int64_t teams = (int64_t)gridDim.x * (threads / 32 / p.warps);
  const int64_t first = (int64_t)blockIdx.x * (threads / 32 / p.warps) + t.index;
  auto fetch = [&](int64_t i, int s) {
    if (i < p.N)
#pragma unroll
      for (int r = 0; r < R; ++r)
        P::fetch(ring + (s * R + r) * slot, elem_at<T>(p.x, i * p.x_ld), team_col<T, A>(t, r), D);
    fetch_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(first + s * teams, s);
  int mine = 0;  // columns of this thread
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = team_col<T, A>(t, r);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = c + P::offset(e) < D;
      mine += in;
      if constexpr (!WS) continue;
      const size_t at = (size_t)(r * E / 4 + e / 4) * threads * 4 + e % 4;
      weight[at] = in ? load_weight(p.weight, p.wbf16, c + P::offset(e), 1.0f) : 0.0f;
      bias[at] = in ? load_weight(p.bias, p.wbf16, c + P::offset(e), 0.0f) : 0.0f;
    }
  }
  const float cols = (float)__reduce_add_sync(~0u, mine);  // of this warp
  int s = 0, parity = 0;
  for (int64_t i = first; i < p.N; i += teams) {
    fetch_wait<S - 1>();
    uint4 raw[R];
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      raw[r] = *reinterpret_cast<const uint4*>(ring + (s * R + r) * slot);
      float f[E];
      Elem<T>::widen(raw[r], f);
      const int c = team_col<T, A>(t, r);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += c + P::offset(e) < D ? f[e] : 0.0f;
    }
    sum = warp_sum(sum);
    fetch(i + S * teams, s);  // the slot has been read
    s = s + 1 == S ? 0 : s + 1;
    const float local = cols > 0.0f ? sum / cols : 0.0f;
    float sq = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[E];
      Elem<T>::widen(raw[r], f);
      const int c = team_col<T, A>(t, r);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = c + P::offset(e) < D ? f[e] - local : 0.0f;
        sq = fmaf(d, d, sq);
      }
    }
    sq = warp_sum(sq);
    float mean = local;
    if (t.warps > 1) {
      float2* now = red + parity * t.warps;
      parity ^= 1;
      if (t.lane == 0) now[t.warp] = make_float2(sum, sq);
      t.meet();
      const float2 o = t.lane < t.warps ? now[t.lane] : make_float2(0.0f, 0.0f);
      mean = warp_sum(o.x) / (float)D;
      // the columns of warp t.lane
      int n = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int left = D - (t.lane + t.warps * r) * 32 * E;
        n += left <= 0 ? 0 : left < 32 * E ? left : 32 * E;
      }
      const float d = t.lane < t.warps && n ? o.x / (float)n - mean : 0.0f;
      sq = warp_sum(fmaf((float)n * d, d, o.y));
    }
    const float rstd = rsqrtf(sq / (float)D + p.eps);
    char* y = elem_at<T>(p.y, i * p.y_ld);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[E], w[E], b[E];
      Elem<T>::widen(raw[r], f);
      const int c = team_col<T, A>(t, r);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = (f[e] - mean) * rstd;
      if constexpr (KEEP)
        keep8<T, A>(f, c, (t.warp + t.warps * r) * (32 * E / kBlock8), D,
                    p.codes + i * p.codes_ld, p.scales + i * ((D + kBlock8 - 1) / kBlock8));
      if constexpr (WS) {
        read_slots<E>(weight + (size_t)r * E * threads, threads, w);
        read_slots<E>(bias + (size_t)r * E * threads, threads, b);
      } else {
        read_weight<T, A>(p.weight, p.wbf16, c, D, 1.0f, w);
        read_weight<T, A>(p.bias, p.wbf16, c, D, 0.0f, b);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf(f[e], w[e], b[e]);
      P::store(y, c, D, f);
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
// [thread] of 2 fp32; the weight [r][k][thread] of 4 fp32; and the teams'
// partial sums.
template <typename T, int A, int R, bool KEPT>
__global__ void __launch_bounds__(512, 1) vc_norm_grad_rows(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Pieces<T, A>;
  constexpr int E = P::E, S = norm_stages(R, true);
  constexpr bool WS = norm_keeps_weight(R);
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
  float* weight = reinterpret_cast<float*>(smem + S * stage) + tid * 4;
  float2* red = reinterpret_cast<float2*>(smem + S * stage + (WS ? R * E * 4 * threads : 0)) +
                t.index * 2 * t.warps;

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
  // columns past the row's end are never fetched: their gradient stays 0
  for (int k = 0; k < S * stage; k += threads * 16)
    if (k + tid * 16 < S * stage) *reinterpret_cast<uint4*>(smem + k + tid * 16) = make_uint4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(first + s * teams, s);
#pragma unroll
  for (int r = 0; r < (WS ? R : 0); ++r) {
    const int c = team_col<T, A>(t, r);
#pragma unroll
    for (int e = 0; e < E; ++e)
      weight[(size_t)(r * E / 4 + e / 4) * threads * 4 + e % 4] =
          c + P::offset(e) < D ? load_weight(p.weight, p.wbf16, c + P::offset(e), 1.0f) : 0.0f;
  }
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
    const float mean = stat.x, rstd = stat.y;
    uint4 graw[R], xraw[R];
    float2 scale[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      graw[r] = *reinterpret_cast<const uint4*>(gslot + at + r * threads * 16);
      if constexpr (KEPT) {
        const char* from = xslot + at + r * threads * E;
        if constexpr (A < E) {
          from -= t.lane * (E - A);  // this lane's first column
          uint32_t word[2] = {0u, 0u};
#pragma unroll
          for (int e = 0; e < E; ++e)
            word[e / 4] |= (uint32_t)(uint8_t)from[P::offset(e)] << (8 * (e % 4));
          xraw[r].x = word[0];
          xraw[r].y = word[1];
        } else if constexpr (E == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(from);
          xraw[r].x = v.x;
          xraw[r].y = v.y;
        } else {
          xraw[r].x = *reinterpret_cast<const uint32_t*>(from);
        }
        scale[r] = *reinterpret_cast<const float2*>(cslot + at + r * threads * 8);
      } else {
        xraw[r] = *reinterpret_cast<const uint4*>(xslot + at + r * threads * 16);
      }
    }
    auto normal = [&](int r, float (&h)[E]) {
      if constexpr (KEPT) {
        const uint32_t word[2] = {xraw[r].x, xraw[r].y};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float sc = SC == 2 && P::offset(e) >= kBlock8 ? scale[r].y : scale[r].x;
          h[e] = code_value(word[e / 4], e % 4) * sc;
        }
      } else {
        Elem<T>::widen(xraw[r], h);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = (h[e] - mean) * rstd;
      }
    };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[E], h[E], w[E];
      Elem<T>::widen(graw[r], f);
      normal(r, h);
      if constexpr (WS) read_slots<E>(weight + (size_t)r * E * threads, threads, w);
      else read_weight<T, A>(p.weight, p.wbf16, team_col<T, A>(t, r), D, 1.0f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dw[r][e] = fmaf(f[e], h[e], dw[r][e]);
        db[r][e] += f[e];
        const float g = f[e] * w[e];
        s1 += g;
        s2 = fmaf(g, h[e], s2);
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
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
    s1 /= (float)D;
    s2 /= (float)D;
    char* dx = elem_at<T>(p.y, i * p.y_ld);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[E], h[E], w[E];
      Elem<T>::widen(graw[r], f);
      normal(r, h);
      if constexpr (WS) read_slots<E>(weight + (size_t)r * E * threads, threads, w);
      else read_weight<T, A>(p.weight, p.wbf16, team_col<T, A>(t, r), D, 1.0f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = (fmaf(f[e], w[e], -s1) - h[e] * s2) * rstd;
      P::store(dx, team_col<T, A>(t, r), D, f);
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
