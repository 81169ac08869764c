// Layer norm kernels for bf16 rows.
#include "norm_rows.cuh"

namespace vcoll {

namespace {

template <int A, bool KEEP>
const void* forward(int chunks) {
  switch (chunks) {
    case 1: return (const void*)&vc_norm_rows<__nv_bfloat16, A, 1, KEEP>;
    case 2: return (const void*)&vc_norm_rows<__nv_bfloat16, A, 2, KEEP>;
    case 4: return (const void*)&vc_norm_rows<__nv_bfloat16, A, 4, KEEP>;
    default: return (const void*)&vc_norm_rows<__nv_bfloat16, A, 8, KEEP>;
  }
}
template <int A, bool KEPT>
const void* backward(int chunks) {
  switch (chunks) {
    case 1: return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 1, KEPT>;
    case 2: return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 2, KEPT>;
    default: return (const void*)&vc_norm_grad_rows<__nv_bfloat16, A, 4, KEPT>;
  }
}
template <int A>
const void* by_pass(int chunks, bool grad, bool kept) {
  if (grad) return kept ? backward<A, true>(chunks) : backward<A, false>(chunks);
  return kept ? forward<A, true>(chunks) : forward<A, false>(chunks);
}

}  // namespace

const void* norm_rows_kernel_bf16(int access, int chunks, bool grad, bool kept) {
  if (access == 8) return by_pass<8>(chunks, grad, kept);
  if (access == 2) return by_pass<2>(chunks, grad, kept);
  return by_pass<1>(chunks, grad, kept);
}

}  // namespace vcoll
