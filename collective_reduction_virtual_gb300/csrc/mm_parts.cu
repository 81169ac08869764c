// The passes around the products of mm_kernels.cu: operands laid out as bf16
// parts, the join of the loss's tiles, and the element-wise gradient of a gated
// block.  All are bound by memory: each value is read and written once, eight
// adjacent ones a thread.
#include "mm_epilogue.cuh"

namespace vcoll {

namespace {

constexpr int kThreads = 256;

// row and group of eight columns of item e; 64-bit division only where needed
__device__ __forceinline__ void item_at(int64_t e, int64_t groups, int64_t& row, int64_t& group) {
  if ((uint64_t)e <= 0xFFFFFFFFull && (uint64_t)groups <= 0xFFFFFFFFull) {
    row = (uint32_t)e / (uint32_t)groups;
    group = (uint32_t)e - (uint32_t)row * (uint32_t)groups;
  } else {
    row = e / groups;
    group = e - row * groups;
  }
}

// Values i .. i + 7 of a matrix of fp32 or bf16, those from `count` on as zeros.
__device__ __forceinline__ void load8(const void* p, int f32, bool load16, int64_t i, int64_t count,
                                      float (&v)[8]) {
  if (f32) {
    const float* q = static_cast<const float*>(p) + i;
    if (load16 && count >= 8) {
      const uint4 a = ld_stream(q), b = ld_stream(q + 4);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < count ? q[j] : 0.0f;
    }
    return;
  }
  const uint16_t* q = static_cast<const uint16_t*>(p) + i;
  if (count >= 8) {
    uint32_t w[4];
    if (load16) {
      const uint4 a = ld_stream(q);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
      // the words that hold them: each holds at least one of the values
      const uint32_t* x = reinterpret_cast<const uint32_t*>((uintptr_t)q & ~(uintptr_t)3);
      const bool odd = (uintptr_t)q & 2;
      const uint32_t y[5] = {x[0], x[1], x[2], x[3], odd ? x[4] : 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = odd ? __funnelshift_r(y[j], y[j + 1], 16) : y[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) Elem<__nv_bfloat16>::widen2(w[j], v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < count ? Elem<__nv_bfloat16>::widen1(q[j]) : 0.0f;
  }
}

// The parts of eight values, 16 bytes each.  One part alone is the value rounded.
__device__ __forceinline__ void store8(void* dst, int64_t i, int64_t plane, int parts, const float (&v)[8]) {
  uint16_t* to = static_cast<uint16_t*>(dst) + i;
  if (parts == 1) {
    *reinterpret_cast<uint4*>(to) = make_uint4(mm_narrow2(v[0], v[1]), mm_narrow2(v[2], v[3]),
                                               mm_narrow2(v[4], v[5]), mm_narrow2(v[6], v[7]));
    return;
  }
  uint16_t q[8][3];
#pragma unroll
  for (int j = 0; j < 8; ++j) mm_parts(v[j], q[j]);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<uint4*>(to + k * plane) =
        make_uint4(q[0][k] | (uint32_t)q[1][k] << 16, q[2][k] | (uint32_t)q[3][k] << 16,
                   q[4][k] | (uint32_t)q[5][k] << 16, q[6][k] | (uint32_t)q[7][k] << 16);
}

// The largest magnitude of dloss over the rows that count, by one CTA; 1 where it
// is zero or not finite.
__device__ __forceinline__ void largest(const MmPackParams& p) {
  __shared__ float part[kThreads / 32];
  float top = 0.0f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < p.N; i += kThreads) {
    const int64_t t = mm_token(p.targets, p.idx64, i);
    const float g = fabsf(p.dloss[i * p.dloss_step]);
    if (t >= 0 && t < p.V && g > top) top = g;
  }
  for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, part[w]);
  *p.scale = top > 0.0f && top < INFINITY ? top : 1.0f;
}

// A CTA's part of the matrices that are laid out; the first CTA is block 0.
__device__ __forceinline__ void pack(const MmPackParams& p, int64_t block) {
  int which = 0;
  while (which + 1 < kMmPackJobs && block >= p.job[which + 1].first_block) ++which;
  const MmPackJob& j = p.job[which];
  const int64_t groups = (j.cols + 7) / 8;
  for (int64_t e = (block - j.first_block) * kThreads + threadIdx.x; e < j.rows * groups; e += j.blocks * kThreads) {
    int64_t row, group;
    item_at(e, groups, row, group);
    bool keep = true;
    if (j.masked) {
      const int64_t t = mm_token(p.targets, p.idx64, row);
      keep = t >= 0 && t < p.V;
    }
    float v[8];
    load8(j.src, p.src_f32, j.load16, row * j.src_ld + group * 8, keep ? j.cols - group * 8 : 0, v);
    store8(j.dst, row * j.dst_ld + group * 8, j.plane, p.parts, v);
  }
}

}  // namespace

// Operands that TMA cannot take as they lie (fp32, odd rows, x of padded tokens) to
// bf16 parts in rows of whole lines; several matrices in one launch, the CTAs
// shared out by their sizes.  50.8e6 + 2.0e6 bf16 values of 1001 columns, 2-byte
// aligned: 44 us, 4.7 TB/s; 16.8e6 of 4096 columns 16 us, 4.2 TB/s.  Odd rows are
// read in the words that hold them, 20 bytes for 16.
__global__ void __launch_bounds__(kThreads) vc_mm_pack(const __grid_constant__ MmPackParams p) {
  pdl_enter();
  if (!p.scale)
    pack(p, blockIdx.x);
  else if (blockIdx.x)
    pack(p, (int64_t)blockIdx.x - 1);
  else
    largest(p);
}

// What a table's gradient is added to, as the first of the fp32 sums that its blocks
// of rows add to.  Once for a piece of the vocabulary: a thousandth of its products.
__global__ void __launch_bounds__(kThreads) vc_mm_widen(const __grid_constant__ MmWidenParams p) {
  pdl_enter();
  const int64_t groups = (p.cols + 7) / 8;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < p.rows * groups; e += p.blocks * kThreads) {
    int64_t row, group;
    item_at(e, groups, row, group);
    float v[8];
    load8(p.src, p.src_f32, p.load16, row * p.src_ld + group * 8, p.cols - group * 8, v);
    float* to = p.dst + row * p.dst_ld + group * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (group * 8 + j < p.cols) to[j] = v[j];
  }
}

// lse[i] = log of the sum over the tiles' (maximum, sum of exponentials), which are
// joined pair by pair: s = s1 e^(m1 - m) + s2 e^(m2 - m) with m the larger maximum.
// A CTA for 32 rows, a warp for every 32nd tile of them.
// Bound by latency: 7 rows of 125 tiles 5.9 us, 8192 rows of 500 16 us (2 TB/s).
__global__ void __launch_bounds__(kMmJoinThreads) vc_mm_join(const __grid_constant__ MmJoinParams p) {
  pdl_enter();
  constexpr int WARPS = kMmJoinThreads / 32;
  __shared__ float2 part[kMmJoinThreads];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  auto add = [&](float2 q) {
    const float top = fmaxf(m, q.x);
    if (fabsf(top) == INFINITY)  // nothing yet but what has no exponential, or NaN; or lse is infinite
      s += q.y;
    else
      s = s * mm_exp(m - top) + q.y * mm_exp(q.x - top);
    m = top;
  };
  if (row < p.N) {
    if (warp == 0 && !p.first) add(p.state[row]);
#pragma unroll 4
    for (int64_t t = warp; t < p.tiles; t += WARPS) add(p.part[t * p.N + row]);
  }
  for (int half = WARPS / 2; half; half /= 2) {
    if (warp >= half && warp < 2 * half) part[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    if (warp < half) add(part[threadIdx.x + half * 32]);
  }
  if (warp || row >= p.N) return;
  if (!p.last) {
    p.state[row] = make_float2(m, s);
    return;
  }
  const int64_t t = mm_token(p.targets, p.idx64, row);
  const float above = logf(s);  // no token at all: log 0
  p.lse[row] = m + above;
  p.loss[row] = t >= 0 && t < p.V ? (m - p.loss[row]) + above : 0.0f;  // of a sure token without lse's rounding
}

// dgate = dh * up * act'(gate), dup = dh * act(gate), next to each other in a row:
// dx sums over both.  16384 x 11008 bf16, silu: 341 us for 1.8 GB, 5.3 TB/s (with the
// exact gelu's erf and for odd rows instructions bound it: 3001 x 2671 19 us, 4.2 TB/s).
// The CTAs behind lay out x and the weights: a launch of its own for that took 4.5 us
// more of 512 x 320 x 1280, 5 of 3001 x 1001 x 2671.
template <int ACT>
__global__ void __launch_bounds__(kThreads) vc_mm_gated_grad(const __grid_constant__ MmGatedGradParams p) {
  pdl_enter();
  if (blockIdx.x >= p.blocks) {
    pack(p.pack, blockIdx.x - p.blocks);
    return;
  }
  const int64_t groups = p.half / 8;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < p.N * groups; e += p.blocks * kThreads) {
    int64_t row, group;
    item_at(e, groups, row, group);
    const int64_t col = group * 8, left = p.F - col;  // what pads a row is zeros: it stands in the sum of dx
    float dh[8], g[8], u[8];
    load8(p.dh, p.f32, p.load16, row * p.dh_ld + col, left, dh);
    load8(p.gate, p.f32, p.load16, row * p.gate_ld + col, left, g);
    load8(p.up, p.f32, p.load16, row * p.up_ld + col, left, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s, ds;
      mm_act(ACT, g[j], s, ds);
      u[j] = dh[j] * u[j] * (s + mm_finite(g[j]) * ds);
      dh[j] = dh[j] * (mm_low(g[j]) * s);
    }
    store8(p.dst, row * p.dst_ld + col, p.plane, p.parts, u);
    store8(p.dst, row * p.dst_ld + p.half + col, p.plane, p.parts, dh);
  }
}

const void* mm_pack_kernel() { return (const void*)vc_mm_pack; }
const void* mm_widen_kernel() { return (const void*)vc_mm_widen; }
const void* mm_join_kernel() { return (const void*)vc_mm_join; }
const void* mm_gated_grad_kernel(int act) {
  return act == VCOLL_SILU   ? (const void*)vc_mm_gated_grad<VCOLL_SILU>
         : act == VCOLL_GELU ? (const void*)vc_mm_gated_grad<VCOLL_GELU>
                             : (const void*)vc_mm_gated_grad<VCOLL_GELU_TANH>;
}

}  // namespace vcoll
