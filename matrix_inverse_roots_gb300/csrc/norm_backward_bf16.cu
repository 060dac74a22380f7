// The norm's backward pass for bf16.
#include "norm_backward.cuh"

namespace dash {

dash_status norm_backward_bf16(const NormBwdArgs& a, const BwdPlan& b, float* part,
                             cudaStream_t st) {
  return backward_c<__nv_bfloat16>(a, b, part, st);
}

int norm_bf16_read_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_dash_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_dash_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

}  // namespace dash
