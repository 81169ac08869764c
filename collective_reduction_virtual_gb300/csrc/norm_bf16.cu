// Layer norm kernels for bf16 rows.
#include "norm_narrow.cuh"
#include "norm_rows.cuh"

namespace vcoll {

namespace {

template <int A, bool KEEP>
const void* forward(int chunks, int threads) {
  if (chunks == 2 && threads <= 256) return (const void*)&vc_norm_rows<__nv_bfloat16, A, 2, 256, KEEP>;
  if (chunks == 4 && threads <= 256) return (const void*)&vc_norm_rows<__nv_bfloat16, A, 4, 256, KEEP>;
  if (chunks == 4 && threads <= 512) return (const void*)&vc_norm_rows<__nv_bfloat16, A, 4, 512, KEEP>;
  if (chunks == 8 && threads <= 512) return (const void*)&vc_norm_rows<__nv_bfloat16, A, 8, 512, KEEP>;
  return nullptr;
}
template <int A, bool KEPT>
const void* backward(int chunks, int threads) {
  if (chunks == 2 && threads <= 256) return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 2, 256, KEPT>;
  if (chunks == 2 && threads <= 512) return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 2, 512, KEPT>;
  if (chunks == 4 && threads <= 512) return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 4, 512, KEPT>;
  return nullptr;
}
template <int A>
const void* by_pass(int chunks, int threads, bool grad, bool kept) {
  if (grad) return kept ? backward<A, true>(chunks, threads) : backward<A, false>(chunks, threads);
  return kept ? forward<A, true>(chunks, threads) : forward<A, false>(chunks, threads);
}

}  // namespace

const void* norm_rows_kernel_bf16(int access, int chunks, int threads, bool grad, bool kept) {
  if (access == 8) return by_pass<8>(chunks, threads, grad, kept);
  if (access == 2) return by_pass<2>(chunks, threads, grad, kept);
  return by_pass<1>(chunks, threads, grad, kept);
}

const void* norm_narrow_kernel_bf16(int access, int lanes, bool grad, bool kept) {
  if (access == 8) return narrow_kernel<__nv_bfloat16, 8>(lanes, grad, kept);
  if (access == 2) return narrow_kernel<__nv_bfloat16, 2>(lanes, grad, kept);
  return narrow_kernel<__nv_bfloat16, 1>(lanes, grad, kept);
}

}  // namespace vcoll
