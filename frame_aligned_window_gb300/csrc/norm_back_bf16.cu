// Gradients of a block's norms: the bf16 kernels.
#include "norm_back.cuh"

namespace wsattn {

cudaError_t norm_backward_bf16(const NormParams& p, bool stream_f32, cudaStream_t s) {
  return stream_f32 ? norm::backward<__nv_bfloat16, float>(p, s) : norm::backward<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace wsattn
