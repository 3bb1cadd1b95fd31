// Gradients of a block's norms: the fp16 kernels.
#include "norm_back.cuh"

namespace wsattn {

cudaError_t norm_backward_fp16(const NormParams& p, bool stream_f32, cudaStream_t s) {
  return stream_f32 ? norm::backward<__half, float>(p, s) : norm::backward<__half, __half>(p, s);
}

}  // namespace wsattn
