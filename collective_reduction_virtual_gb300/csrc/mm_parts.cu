// The passes around the products of mm_kernels.cu: operands laid out as bf16
// parts, the join of the loss's tiles, the scale of the loss's gradient, and the
// element-wise gradient of a gated block.
#include "mm_epilogue.cuh"

namespace vcoll {

namespace {
constexpr int kThreads = 256;
}

// dst[part][i][j]: the parts of src[i][j], a thread for 4 columns.  Reads 2 or 4
// bytes a value and writes 2 or 6: bound by memory.
__global__ void __launch_bounds__(kThreads) vc_mm_pack(const __grid_constant__ MmPackParams p) {
  pdl_enter();
  const int64_t quads = (p.cols + 3) / 4;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < p.rows * quads;
       e += (int64_t)gridDim.x * kThreads) {
    const int64_t i = e / quads, j0 = e % quads * 4;
    bool keep = true;
    if (p.targets) {
      const int64_t t = mm_token(p.targets, p.idx64, i);
      keep = t >= 0 && t < p.V;
    }
    uint16_t q[4][3];
    for (int j = 0; j < 4; ++j) {
      const bool read = keep && j0 + j < p.cols;
      const float x = read ? mm_load(p.src, p.src_f32, i * p.src_ld + j0 + j) : 0.0f;
      mm_parts(x, q[j]);
    }
    for (int k = 0; k < p.parts; ++k)  // rows are padded to 8 values
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dst) + k * p.plane + i * p.dst_ld + j0) =
          make_uint2(q[0][k] | (uint32_t)q[1][k] << 16, q[2][k] | (uint32_t)q[3][k] << 16);
  }
}

// A CTA for 32 rows, a warp for every eighth tile of them.
__global__ void __launch_bounds__(kThreads) vc_mm_join(const __grid_constant__ MmJoinParams p) {
  pdl_enter();
  __shared__ float2 part[kThreads];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  auto add = [&](float2 q) {
    const float top = fmaxf(m, q.x);
    if (top == -INFINITY) {  // nothing yet but what has no exponential, or NaN
      s += q.y;
      return;
    }
    s = s * mm_exp(m - top) + q.y * mm_exp(q.x - top);
    m = top;
  };
  if (row < p.N) {
    if (warp == 0 && !p.first) add(p.state[row]);
    for (int64_t t = warp; t < p.tiles; t += kThreads / 32) add(p.part[t * p.N + row]);
  }
  part[threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (warp || row >= p.N) return;
  for (int w = 1; w < kThreads / 32; ++w) add(part[w * 32 + lane]);
  if (!p.last) {
    p.state[row] = make_float2(m, s);
    return;
  }
  const int64_t t = mm_token(p.targets, p.idx64, row);
  const float lse = m + logf(s);  // no token at all: log 0
  p.lse[row] = lse;
  p.loss[row] = t >= 0 && t < p.V ? lse - p.loss[row] : 0.0f;
}

// One CTA.  1 where the largest magnitude is zero or not finite.
__global__ void __launch_bounds__(1024) vc_mm_scale(const __grid_constant__ MmScaleParams p) {
  pdl_enter();
  __shared__ float part[32];
  float top = 0.0f;
  for (int64_t i = threadIdx.x; i < p.N; i += 1024) {
    const int64_t t = mm_token(p.targets, p.idx64, i);
    const float g = fabsf(p.dloss[i * p.step]);
    if (t >= 0 && t < p.V && g > top) top = g;
  }
  for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 32; ++w) top = fmaxf(top, part[w]);
  *p.scale = top > 0.0f && top < INFINITY ? top : 1.0f;
}

// dgate = dh * up * act'(gate), dup = dh * act(gate).
__global__ void __launch_bounds__(kThreads) vc_mm_gated_grad(const __grid_constant__ MmGatedGradParams p) {
  pdl_enter();
  uint16_t* dst = static_cast<uint16_t*>(p.dst);
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < p.N * p.half;
       e += (int64_t)gridDim.x * kThreads) {
    const int64_t i = e / p.half, j = e % p.half;
    float dg = 0.0f, du = 0.0f;
    if (j < p.F) {  // what pads a row stands in the sum of dx
      const float dh = mm_load(p.dh, p.f32, i * p.dh_ld + j), g = mm_load(p.gate, p.f32, i * p.gate_ld + j);
      float s, ds;
      mm_act(p.act, g, s, ds);
      dg = dh * mm_load(p.up, p.f32, i * p.up_ld + j) * (s + g * ds);
      du = dh * (g * s);
    }
    if (p.parts == 1) {  // rounded for the product, as its other operand is
      dst[i * p.dst_ld + j] = Elem<__nv_bfloat16>::narrow1(dg);
      dst[i * p.dst_ld + p.half + j] = Elem<__nv_bfloat16>::narrow1(du);
      continue;
    }
    uint16_t qg[3], qu[3];
    mm_parts(dg, qg);
    mm_parts(du, qu);
    for (int k = 0; k < p.parts; ++k) {
      dst[k * p.plane + i * p.dst_ld + j] = qg[k];
      dst[k * p.plane + i * p.dst_ld + p.half + j] = qu[k];
    }
  }
}

const void* mm_pack_kernel() { return (const void*)vc_mm_pack; }
const void* mm_join_kernel() { return (const void*)vc_mm_join; }
const void* mm_scale_kernel() { return (const void*)vc_mm_scale; }
const void* mm_gated_grad_kernel() { return (const void*)vc_mm_gated_grad; }

}  // namespace vcoll
