// The norms at a block's ends on rows of fp32.
#include "block_norm_kernels.cuh"

namespace gemm_f32_impl {

int block_norm_f32(BlockArgs& a, const BlockLaunch& l) { return forward<float>(a, l); }

int block_norm_grad_f32(BlockGradArgs& a, void* const (&vectors_out)[kSums], const BlockLaunch& l) {
  return gradient<float>(a, vectors_out, l);
}

}  // namespace gemm_f32_impl
