// Private interface of the bfloat16 tensor-core product on CTA pairs
// (half_gemm.cu), used by the vocabulary loss.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "launch.h"

namespace gemm_f32_impl {

// One operand: `parts` stored row-major bfloat16 matrices of rows x cols
// elements with row stride ld, `plane` elements apart, whose sum is the
// operand.  K-major: rows run along M (or N), columns along K.  MN-major:
// the stored matrix is K x M (or K x N).  The base is 16-byte aligned and ld
// and plane are multiples of 8.
struct HalfOperand {
  const void* ptr;
  long long ld;
  long long plane;
  bool mn_major;
};

// What becomes of a finished tile of D = A B^T (D is M x N).
struct HalfGemm {
  int M, N, K;
  int parts;                    // 1, or 3 (fp32 operands split into three parts)
  HalfOperand a, b;
  // -- a stored product: C = *scale * D (+ add)
  void* c = nullptr;
  long long ldc = 0;
  bool c_f32 = false;           // fp32, else bfloat16
  const float* scale = nullptr; // device
  const float* add = nullptr;   // fp32, row stride ldadd; may be c itself
  long long ldadd = 0;
  float* partials = nullptr;    // half_gemm_scratch() bytes
  // -- or logits (c == nullptr): per row and 128 columns the maximum m of z
  // and the sum of 2^((z - m) log2 e); with `exps`, those powers
  // too (fp16 times 2^15 for one part, fp32 for three), zero from column N on
  float2* stats = nullptr;      // [2 ceil(N / 256)][ld_stats]
  long long ld_stats = 0;
  void* exps = nullptr;         // M rows of ld_exps >= 256 ceil(N / 256) elements
  long long ld_exps = 0;
  LossTargets targets = {};     // of its rows
  float* label_logit = nullptr; // per row the logit at its target
  unsigned* arrived = nullptr;  // set to 0, for the kernel that counts arrivals next
  // --
  int num_sms, device;
  unsigned* err;
};

// Bytes of partial tiles that the stored product of this shape needs (0 when
// its last wave is not split along K).
size_t half_gemm_scratch(int M, int N, int K, int parts, int num_sms);

// Returns 0 or a negative GEMM_F32_E* code; counts its kernels in *launches.
int launch_half_gemm(const HalfGemm& g, cudaStream_t stream, int* launches);

// The same two products for few rows (at most kFewRows), where reading w is
// what takes the time (few_gemm.cu).  w is read as it is stored, fp32
// included (f32: its three parts are made on the way to the tensor cores).
// For dx its rows start on 16-byte boundaries; for the logits they may not:
// the rows then fall into classes, and b holds a copy of x for each.
constexpr int kFewRows = 128;     // fp32: the pair kernel would first store w in three parts (64 x 4096
                                  // x 65536 938 us against 249; 128 rows, width x vocabulary: 4096 x
                                  // 65536 942 against 388, 1024 x 32768 131 against 87, 512 x 131072
                                  // 242 against 195, 8192 x 32000 927 against 361)
constexpr int kFewRowsBf16 = 32;  // 4096 x 65536: 103 us against the pair kernel's 158 with one row, 112
                                  // against 110 with 32 (gradients 311 against 322), 117 against 111
                                  // with 64, 138 against 111 with 128; 8192 x 32000 with 32 rows 105
                                  // against 109.  With narrow rows the pair kernel is the better one
                                  // from fewer on: 1024 x 32768 23 against 29 with one, 29 against its 25
                                  // with 32; 512 x 131072 45 against 46 with one, 54 against 43 with 16
constexpr int kFewPiece = 32;     // columns per statistic of its logits

// Rows of w as TMA reads them: every `count`-th row has the same distance
// from a 16-byte boundary, so that class c, the rows c, c + count, ..., is a
// matrix that begins shift(c) elements before row c.  Units of kFewPiece rows
// of a class make the logits' work and statistics: class by class, unit by
// unit, `units` of each.
struct FewClasses {
  int count, units;
  int shift0, step, mask;         // shift(c) = (shift0 + c step) & mask
  bool aligned() const { return count == 1 && shift0 == 0; }
};
constexpr int kFewMostClasses = 8;

FewClasses few_classes(bool f32, const void* w, long long ldw, int vocab);

struct FewGemm {
  bool f32;
  int rows, width, vocab;
  const void* w;                  // vocab x width
  long long ldw;
  HalfOperand b;                  // K-major, rows x (width for logits, vocab for dx)
  // -- logits: as HalfGemm, with statistics per unit.  Unless classes is
  // aligned, b has class c's copy of x (or of its parts) c parts planes on,
  // shift(c) columns to the right between zeros, all b.ld columns of it
  // written; vocab >= classes.count and exps is null.
  FewClasses classes = {};
  float2* stats = nullptr;        // [classes.count units][ld_stats]
  long long ld_stats = 0;
  void* exps = nullptr;
  long long ld_exps = 0;
  LossTargets targets = {};
  float* label_logit = nullptr;
  unsigned* arrived = nullptr;
  // -- or dx = *scale * b w (dx != nullptr); `two`: b's rows are two parts,
  // one below the other, of half as many rows of dx
  void* dx = nullptr;
  bool two = false;
  long long lddx = 0;
  const float* scale = nullptr;
  float* partials = nullptr;      // few_gemm_scratch() bytes
  // --
  int num_sms, device;
  unsigned* err;
};

size_t few_gemm_scratch(int rows, int width, int vocab, int num_sms);   // of dx
int launch_few_gemm(const FewGemm& g, cudaStream_t stream, int* launches);

}  // namespace gemm_f32_impl
