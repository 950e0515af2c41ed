// The norms at a block's ends on rows of bfloat16.
#include "block_norm_kernels.cuh"

namespace gemm_f32_impl {

int block_norm_bf16(BlockArgs& a, const BlockLaunch& l) { return forward<__nv_bfloat16>(a, l); }

int block_norm_grad_bf16(BlockGradArgs& a, void* const (&vectors_out)[kSums], const BlockLaunch& l) {
  return gradient<__nv_bfloat16>(a, vectors_out, l);
}

}  // namespace gemm_f32_impl
