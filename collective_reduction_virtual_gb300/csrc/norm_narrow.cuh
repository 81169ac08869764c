// Layer norm and its gradient for narrow rows, up to 32 * E columns (256 of
// bf16, 128 of fp32: heads, small models), instantiated in norm_f32.cu and
// norm_bf16.cu.
//
// A row is taken by G lanes (8, 16 or 32), so a warp takes 32 / G rows at a
// time, and kNarrowRows times that in one go: the loads of all of them are in
// flight together, and their sums, a few shuffles each, overlap.  Weight and
// bias stay in registers.  What bounds these kernels is the latency of such a
// go; a warp of norm_rows.cuh would spend it on one row, most of its lanes idle
// (100000 x 64 bf16: 25.7 us forward and 30.0 backward; here 7.1 and 10.7).
// 200000 x 128 bf16: 22 us forward, 4.7 TB/s, and 30 backward, 5.2 TB/s.
#pragma once

#include "layers_internal.h"
#include "norm_common.cuh"
#include "row_access.cuh"

namespace vcoll {

template <typename T, int A, int G, bool KEEP>
__global__ void __launch_bounds__(kRowThreads, 3) vc_norm_narrow(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Group<T, A, G>;
  constexpr int E = P::E, U = kNarrowRows, S = 32 / G;
  const P g;
  const int D = (int)p.D;
  float w[E], b[E];
  g.weights(p.weight, p.wbf16, D, 1.0f, w);
  g.weights(p.bias, p.wbf16, D, 0.0f, b);
  const uint32_t rows = (uint32_t)p.N, warps = gridDim.x * (kRowThreads / 32);
  for (uint32_t unit = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); unit * (U * S) < rows; unit += warps) {
    const uint32_t first = unit * (U * S) + g.sub;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first + u * S;
      raw[u] = g.load(elem_at<T>(p.x, i * p.x_ld), D, i < rows);
    }
    float f[U][E], mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Elem<T>::widen(raw[u], f[u]);
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int e = 0; e < E; e += 2) add2(x, y, x, y, f[u][e], f[u][e + 1]);
      mean[u] = P::sum(x + y) / (float)D;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        add2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], -mean[u], -mean[u]);
        if (g.c + P::offset(e) >= D) f[u][e] = 0.0f;
        if (g.c + P::offset(e + 1) >= D) f[u][e + 1] = 0.0f;
        fma2(x, y, f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], x, y);
      }
      rstd[u] = rsqrtf(P::sum(x + y) / (float)D + p.eps);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first + u * S;
#pragma unroll
      for (int e = 0; e < E; e += 2) mul2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], rstd[u], rstd[u]);
      if constexpr (KEEP)
        g.keep(f[u], D, i < rows, p.codes + i * p.codes_ld, p.scales + (int64_t)i * ((D + kBlock8 - 1) / kBlock8));
      if (i >= rows) continue;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        fma2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], w[e], w[e + 1], b[e], b[e + 1]);
      g.store(elem_at<T>(p.y, i * p.y_ld), D, f[u]);
      if (g.c == 0) {
        if (p.mean) p.mean[i] = mean[u];
        if (p.rstd) p.rstd[i] = rstd[u];
      }
    }
  }
}

template <typename T, int A, int G, bool KEPT>
__global__ void __launch_bounds__(kRowThreads, 2) vc_norm_grad_narrow(const __grid_constant__ NormParams p) {
  pdl_enter();
  using P = Group<T, A, G>;
  constexpr int E = P::E, U = kNarrowRows, S = 32 / G, NW = kRowThreads / 32;
  __shared__ float sums[2][NW][G * E];
  const P g;
  const int D = (int)p.D, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[E], dw[E], db[E];
  g.weights(p.weight, p.wbf16, D, 1.0f, w);
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.0f;
  const uint32_t rows = (uint32_t)p.N, warps = gridDim.x * NW;
  for (uint32_t unit = blockIdx.x * NW + warp; unit * (U * S) < rows; unit += warps) {
    const uint32_t first = unit * (U * S) + g.sub;
    uint4 graw[U], xraw[U];
    float h[U][E], mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first + u * S;
      const bool in = i < rows;
      graw[u] = g.load(elem_at<T>(p.grad, i * p.grad_ld), D, in);
      if constexpr (!KEPT) {
        xraw[u] = g.load(elem_at<T>(p.x, i * p.x_ld), D, in);
        mean[u] = in ? p.mean[i] : 0.0f;
      }
      rstd[u] = in ? p.rstd[i] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first + u * S;
      if constexpr (KEPT) {
        g.kept(p.codes + i * p.codes_ld, p.scales + (int64_t)i * ((D + kBlock8 - 1) / kBlock8), D, i < rows, h[u]);
      } else {
        Elem<T>::widen(xraw[u], h[u]);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          add2(h[u][e], h[u][e + 1], h[u][e], h[u][e + 1], -mean[u], -mean[u]);
          mul2(h[u][e], h[u][e + 1], h[u][e], h[u][e + 1], rstd[u], rstd[u]);
        }
        // past the row's end h is -mean * rstd: where that is no finite number, 0
        // times it would reach the row's sum
        if (D < G * E && !isfinite(mean[u] * rstd[u])) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (g.c + P::offset(e) >= D) h[u][e] = 0.0f;
        }
      }
    }
    // columns past the row's end, and rows past the last, have a gradient of 0
    float f[U][E], s1[U], s2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Elem<T>::widen(graw[u], f[u]);
      float ax = 0.0f, ay = 0.0f, bx = 0.0f, by = 0.0f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        fma2(dw[e], dw[e + 1], f[u][e], f[u][e + 1], h[u][e], h[u][e + 1], dw[e], dw[e + 1]);
        add2(db[e], db[e + 1], db[e], db[e + 1], f[u][e], f[u][e + 1]);
        mul2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], w[e], w[e + 1]);
        add2(ax, ay, ax, ay, f[u][e], f[u][e + 1]);
        fma2(bx, by, f[u][e], f[u][e + 1], h[u][e], h[u][e + 1], bx, by);
      }
      s1[u] = P::sum(ax + ay) / -(float)D;
      s2[u] = P::sum(bx + by) / -(float)D;
    }
    if (!p.y) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first + u * S;
      if (i >= rows) continue;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        add2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], s1[u], s1[u]);
        fma2(f[u][e], f[u][e + 1], h[u][e], h[u][e + 1], s2[u], s2[u], f[u][e], f[u][e + 1]);
        mul2(f[u][e], f[u][e + 1], f[u][e], f[u][e + 1], rstd[u], rstd[u]);
      }
      g.store(elem_at<T>(p.y, i * p.y_ld), D, f[u]);
    }
  }
  if (!p.part) return;
  // the groups of a warp, then its warps, in order
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int d = G; d < 32; d *= 2) {
      dw[e] += __shfl_xor_sync(~0u, dw[e], d);
      db[e] += __shfl_xor_sync(~0u, db[e], d);
    }
    if (lane < G) {
      sums[0][warp][g.c + P::offset(e)] = dw[e];
      sums[1][warp][g.c + P::offset(e)] = db[e];
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * D; k += kRowThreads) {
    const int which = k >= D, at = k - which * D;
    float s = 0.0f;
    for (int n = 0; n < NW; ++n) s += sums[which][n][at];
    p.part[(size_t)(blockIdx.x * 2 + which) * D + at] = s;
  }
}

// access: elements of an access; lanes: of a row
template <typename T, int A, int G>
const void* narrow_kernel(bool grad, bool kept) {
  if (grad) return kept ? (const void*)&vc_norm_grad_narrow<T, A, G, true> : (const void*)&vc_norm_grad_narrow<T, A, G, false>;
  return kept ? (const void*)&vc_norm_narrow<T, A, G, true> : (const void*)&vc_norm_narrow<T, A, G, false>;
}
template <typename T, int A>
const void* narrow_kernel(int lanes, bool grad, bool kept) {
  return lanes == 8    ? narrow_kernel<T, A, 8>(grad, kept)
         : lanes == 16 ? narrow_kernel<T, A, 16>(grad, kept)
                       : narrow_kernel<T, A, 32>(grad, kept);
}

}  // namespace vcoll
