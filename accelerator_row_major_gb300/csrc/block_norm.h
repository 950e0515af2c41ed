// Private interface of the norms at a block's ends: how their rows are laid
// out over threads and shared memory, and what the kernels are given
// (block_norm.cu checks, block_plan.h lays rows out, block_norm_f32.cu and
// block_norm_bf16.cu hold the kernels of one type each).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gemm_f32_block.h"

namespace gemm_f32_impl {

constexpr int kRowWarps = 16;            // that compute, at most
constexpr int kProducers = 4;            // warps that fill the ring, at most
constexpr int kProducerThreads = 32 * kProducers;
constexpr int kMostCtas = 8;             // of a cluster
constexpr int kStats = 4;                // per row: mean and rstd of h, of the branch
constexpr int kMostChunk = 8;            // rows of a stage, where all rows lie one behind the other
constexpr int kMostLoose = 4;            // and where they do not
constexpr int kSliceUnit = 512;          // columns: their exponents fill 16 bytes

// Bytes of `cols` columns of a matrix whose elements take `size` (0: exponents).
__host__ __device__ inline uint32_t source_bytes(int size, int cols) {
  return size ? static_cast<uint32_t>(size) * cols
              : static_cast<uint32_t>(cols + GEMM_F32_SAVED_BLOCK - 1) / GEMM_F32_SAVED_BLOCK;
}

// One matrix that a row is read from.  size: bytes per element, or 0 for the
// exponents of 8-bit rows (a byte per 32 columns).
struct RowSource {
  const char* p;                         // null: not there
  const char* end;                       // one past the last byte that may be read
  long long ld;                          // bytes from row to row
  int size;
  uint32_t at;                           // of its chunk within a stage
  uint32_t pitch;                        // there, from row to row: ld where `packed`
  int packed;                            // rows one behind the other: a chunk is one copy
};

// How a launch lays out its rows.
struct RowPlan {
  int width, slice;                      // columns of a row, of a CTA's part
  int lanes, groups, stages, ctas;
  int turn;                              // rows of all groups at a time
  int chunk;                             // rows of a stage: of whole groups, a divisor of turn
  int producers;                         // 4, 2 or 1, a divisor of stages
  uint32_t stage_bytes;
  uint32_t ring_at;                      // in dynamic shared memory, behind the weights
  uint32_t bars_at;                      // the ring's barriers: behind it and behind the groups' sums that take its place,
                                         // since producers may still be at their last waits then
  uint32_t stats_at;                     // of the rows' statistics within a stage; 0: they do not come this way
  long long rows;
};

// Vectors over the columns, by their place in VectorArgs.
enum { kWeight, kBias, kPostWeight, kPostBias, kGateVector, kVectors };

struct VectorArgs {
  const void* p[kVectors];               // null where `there`: the default
  int slot[kVectors];                    // of the vectors in shared memory, -1: not there
  int f32;
  int joined;                            // the post weight's place holds it times the gate
};

enum { kNoGate, kChannelGate, kElementGate };

// Matrices of the forward pass and of the gradient.
enum { kInBranch, kInResidual, kInGate, kInputs };
enum { kGradDy, kGradDh, kGradH, kGradHExponents, kGradBranch, kGradBranchExponents, kGradGate, kGradInputs };

// Vectors' gradients.
enum { kSumWeight, kSumBias, kSumGate, kSumPostWeight, kSumPostBias, kSums };

struct Output {
  void* p;                               // null: not wanted
  long long ld;
};

struct BlockArgs {
  RowPlan plan;
  RowSource in[kInputs];
  VectorArgs vectors;
  int rms, post, gate;
  float eps, alpha, beta;
  Output y, h;
  float* stats;
  unsigned* err;
};

struct BlockGradArgs {
  RowPlan plan;
  RowSource in[kGradInputs];
  VectorArgs vectors;
  int rms, post, gate, branch;           // branch: it is read
  float alpha, beta;
  const float* stats;
  Output dbranch, dresidual, dgate;      // dgate: of a matrix
  float* partials;                       // [CTA or cluster][sums][ld_partials]
  long long ld_partials;                 // width rounded up to 4
  int sum[kSums];                        // a vector's place in the partials, -1: not wanted
  int sums;
  unsigned* err;
};

// The forward call or the gradient on rows of one type: picks the kernel, lays
// the rows out and launches.  `vectors`: how many lie in shared memory;
// `aligned`: all rows are whole 16-byte vectors on 16-byte boundaries.
struct BlockLaunch {
  int vectors;
  bool aligned, weights_f32;
  int device, num_sms;
  cudaStream_t stream;
  int* launches;
  const char** kernel;
};

int block_norm_f32(BlockArgs& a, const BlockLaunch& l);
int block_norm_bf16(BlockArgs& a, const BlockLaunch& l);
int block_norm_grad_f32(BlockGradArgs& a, void* const (&vectors_out)[kSums], const BlockLaunch& l);
int block_norm_grad_bf16(BlockGradArgs& a, void* const (&vectors_out)[kSums], const BlockLaunch& l);

}  // namespace gemm_f32_impl
