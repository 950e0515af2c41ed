// Softmax cross entropy over a vocabulary, with its gradients (sm_103a).
//
//   z = x w^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   g = exp(z - lse) - onehot(y),  dx = s g w,  dw = s g^T x
//
// The logits are a product of 2 T V D operations whose result is only needed
// through its rows' maxima and sums of exponentials, so its epilogue
// (half_gemm.cu) reduces each 128 columns to a maximum m and a sum of
// exponentials relative to m, and the rows join these:
//   M = max m_i,  S = sum s_i exp(m_i - M),  lse = M + log S.
// What bounds it: few rows, the read of w; many rows, the tensor cores.
//
// With gradients the logits are computed once too (6 T V D operations in
// all, not 8): for a piece of the rows at a time the epilogue keeps
// e = exp(z - m), the rescaling pass turns it in place into
//   g = e exp(m - M) / S - onehot
// and two more products give dx = s g w and dw += s g^T x.  e is kept in
// fp16 (times 2^15: 11 bits for whatever lies within 2^-29 of its tile's
// maximum, which itself is exact) and g in bfloat16, the operand type of the
// products: one rounding of g, by up to 2^-8 of it (at a target of small
// probability p that is the p of g = p - 1 up to 2^-9).  It is of the size of
// the rounding of the results, and adds to it where few terms make an element:
// with one part, errors against 64 bits over those of products with g in fp32
// measured 1.42 for dw of one row x 4096 x 65536, 1.07 for 8 x 512 x 4096, 1.02
// from 32 rows on, 1.00 for 1001 x 777 x 32001.  So few rows (few_gemm.cu) hold
// g in two parts, the second what the rounding left, one below the other as
// twice as many rows of g (and of x, for dw): dx is the sum of a pair of rows.
// With more rows that would double two of the three products.  The row scale s
// is applied in fp32 to the finished sums.  fp32 operands keep e in fp32 and g
// as three bfloat16 parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_f32_lm.h"
#include "device_common.cuh"
#include "half_gemm.h"
#include "launch.h"
#include "row_common.cuh"
#include "workspace.h"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

using bf16 = __nv_bfloat16;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPieceBits = 7;                       // 128 columns per statistic,
constexpr int kFewPieceBits = 5;                    // 32 with few rows
static_assert(1 << kFewPieceBits == kFewPiece, "columns per statistic");
constexpr size_t kDefaultPieceBytes = size_t{4} << 30;
constexpr size_t kMostStatsBytes = size_t{256} << 20;

// What a call computes for its own later kernels.
struct Factors {
  float grad;      // s: grad_scale, divided for the mean
};

// ---------------------------------------------------------------- joining
// lse and loss of 4 rows per CTA (4 statistics of a piece share a 32-byte
// sector): the largest maximum M of a row's pieces, then S = sum s exp(m - M).
// A piece with sum 0 has nothing above -inf (its m is that) and does not
// count; a NaN sum does.  joined (may be null) receives (M, 1 / S).
//
// The CTA that finishes last adds up what the call needs of all rows: the
// factors (in the first piece of the rows) and the total (in the last), from
// the CTAs' partial sums in a fixed order.
constexpr int kJoinRows = 4;
constexpr int kJoinThreads = 256;      // 1024 where the rows alone leave SMs idle
constexpr int kJoinThreadsFew = 1024;

struct JoinArgs {
  const float2* stats;
  long long ld;
  int pieces, rows;
  LossTargets targets;       // of these rows, as what follows
  const float* label_logit;
  float* loss;
  float* lse;
  float2* joined;
  float* sums;               // per CTA: its rows' losses, and how many count
  int* counts;
  // the whole call
  LossTargets all_targets;
  int all_rows;
  const float* all_sums;
  const int* all_counts;
  bool first, last, mean;
  float grad_scale;
  Factors* factors;
  float* total;
  unsigned* arrived;         // set to 0 by the logits' kernel
  unsigned* err;
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS) loss_join_kernel(const JoinArgs a) {
  constexpr int kChains = THREADS / kJoinRows, kWarps = THREADS / 32;
  __shared__ float tops[kWarps][kJoinRows], sums[kWarps][kJoinRows];
  __shared__ float part_sum[kWarps];
  __shared__ int part_count[kWarps];
  __shared__ bool finish;
  grid_launch_dependents();
  grid_dependency_wait();
  const int r = threadIdx.x % kJoinRows, chain = threadIdx.x / kJoinRows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kJoinRows + r;
  const float2* const mine = a.stats + row;
  const int end = row < a.rows ? a.pieces : 0;
  // this row's label and logit, for the lanes that finish it: loaded first,
  // under the statistics
  const bool finisher = warp == 0 && lane < kJoinRows && row < a.rows;
  int label = -1;
  float logit = 0.0f;
  if (finisher) {
    label = label_at(a.targets, row);
    logit = a.label_logit[row];       // of a row that does not count: not used
  }
  float top = -INFINITY;
#pragma unroll 8
  for (int i = chain; i < end; i += kChains) {
    const float2 p = __ldg(mine + i * a.ld);
    top = p.y != 0.0f ? fmaxf(top, p.x) : top;
  }
#pragma unroll
  for (int o = kJoinRows; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane < kJoinRows) tops[warp][lane] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w][r]);
  float sum = 0.0f;
#pragma unroll 8
  for (int i = chain; i < end; i += kChains) {
    const float2 p = __ldg(mine + i * a.ld);
    sum += p.y != 0.0f ? p.y * exp2f((p.x - top) * kLog2e) : 0.0f;
  }
#pragma unroll
  for (int o = kJoinRows; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane < kJoinRows) sums[warp][lane] = sum;
  __syncthreads();
  float s = 0.0f;
  int n = 0;
  if (warp == 0) {
    if (finisher) {
      sum = sums[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) sum += sums[w][r];
      const float l = sum == 0.0f ? -INFINITY : fmaf(kLn2, log2f(sum), top);
      if (label >= 0) {
        s = l - logit;
      } else {
        const long long y = a.targets.bits == 64 ? static_cast<const long long*>(a.targets.p)[row]
                                                 : static_cast<const int*>(a.targets.p)[row];
        if (y != a.targets.ignore) record_error(a.err + 1, kSiteTarget);
      }
      if (a.lse) a.lse[row] = l;
      if (a.loss) a.loss[row] = s;
      if (a.joined) a.joined[row] = make_float2(top, 1.0f / sum);
    }
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
    n = __popc(__ballot_sync(0xFFFFFFFFu, label >= 0));
  }
  if (a.all_rows > kJoinRows) {         // else this CTA has all of them
    if (threadIdx.x == 0) {
      a.sums[blockIdx.x] = s;
      a.counts[blockIdx.x] = n;
      __threadfence();
      finish = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!finish) return;
    __threadfence();
    // ---- the last CTA
    if (!a.first && !a.last) return;
    s = 0.0f;
    n = 0;
    if (a.first && !a.last) {           // later pieces of the rows are not joined yet
#pragma unroll 8
      for (unsigned t = threadIdx.x; t < static_cast<unsigned>(a.all_rows); t += THREADS)
        n += label_at(a.all_targets, t) >= 0;
    } else {
      const int groups = (a.all_rows - 1) / kJoinRows + 1;
#pragma unroll 4
      for (int i = threadIdx.x; i < groups; i += THREADS) {
        s += __ldcg(a.all_sums + i);
        n += __ldcg(a.all_counts + i);
      }
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    float v[1] = {s};
    warp_sum<1>(v);
    if (lane == 0) {
      part_sum[warp] = v[0];
      part_count[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
      v[0] = lane < kWarps ? part_sum[lane] : 0.0f;
      warp_sum<1>(v);
      s = v[0];
      n = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? part_count[lane] : 0);
    }
  }
  if (threadIdx.x != 0) return;
  const float per = a.mean ? static_cast<float>(n > 1 ? n : 1) : 1.0f;
  if (a.first && a.factors) a.factors->grad = a.grad_scale / per;
  if (a.last && a.total) *a.total = s / per;
}

// The rescaling pass of the gradient, g = e exp(m - M) / S - onehot: 4 rows by
// a band of the columns per CTA.
constexpr int kRescaleThreads = 256;
constexpr int kRescaleRows = 4;

// How e is held: fp32, or fp16 bits.
template <int PARTS>
struct Exps {
  using type = float;
  static __device__ __forceinline__ float value(const Raw<float, 8>& r, int j) { return r.at(j); }
};
template <>
struct Exps<1> {
  using type = uint16_t;
  static __device__ __forceinline__ float value(const Raw<uint16_t, 8>& r, int j) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(r.w[j >> 1] >> (16 * (j & 1)))));
  }
};

template <int PARTS>
__global__ void __launch_bounds__(kRescaleThreads)
    loss_rescale_kernel(const float2* stats, long long ld_stats, int piece_bits, const float2* joined,
                        int rows, int cols, unsigned band, LossTargets targets, void* exps, long long ld,
                        bf16* parts, long long plane, bool two, unsigned* err) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int row0 = blockIdx.x * kRescaleRows;
  [[maybe_unused]] const size_t extent = static_cast<size_t>(rows) * ld;
  int label[kRescaleRows];
  float m[kRescaleRows], inv[kRescaleRows];
#pragma unroll
  for (int r = 0; r < kRescaleRows; ++r) {
    const int row = min(row0 + r, rows - 1);
    const float2 j = __ldg(joined + row);
    label[r] = label_at(targets, row);
    m[r] = j.x;
    inv[r] = j.y * (PARTS == 3 ? 1.0f : 1.0f / 32768.0f);
  }
  // unsigned: a step beyond the last column does not pass the type's end
  const unsigned c_end = min(static_cast<unsigned>(cols), (blockIdx.y + 1u) * band);
  for (unsigned c = blockIdx.y * band + threadIdx.x * 8; c < c_end; c += kRescaleThreads * 8) {
    // the rows' loads first, so that one round trip covers them
    Raw<typename Exps<PARTS>::type, 8> e[kRescaleRows];
    float f[kRescaleRows];
#pragma unroll
    for (int r = 0; r < kRescaleRows; ++r) {
      const size_t at = static_cast<size_t>(row0 + r) * ld + c;
      e[r].zero();
      f[r] = 0.0f;
      if (row0 + r >= rows || !GEMM_IN_EXTENT(at + 7, extent, err, kSiteBoundsScratch)) continue;
      e[r].load_once(static_cast<const typename Exps<PARTS>::type*>(exps) + at);
      f[r] = __ldg(&stats[(c >> piece_bits) * ld_stats + row0 + r].x);
    }
#pragma unroll
    for (int r = 0; r < kRescaleRows; ++r) {
      if (row0 + r >= rows) break;
      const size_t at = static_cast<size_t>(row0 + r) * ld + c;
      if (!GEMM_IN_EXTENT(at + 7, extent, err, kSiteBoundsScratch)) continue;
      const float by = exp2f((f[r] - m[r]) * kLog2e) * inv[r];
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = Exps<PARTS>::value(e[r], j) * by;
        if (static_cast<int>(c) + j == label[r]) g[j] -= 1.0f;
        if (label[r] < 0) g[j] = 0.0f;
      }
      if constexpr (PARTS == 3) {
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          store_vec<bf16, 8>(parts + part * plane + at, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] -= __bfloat162float(__float2bfloat16_rn(g[j]));
        }
      } else {
        store_vec<bf16, 8>(static_cast<bf16*>(exps) + at, g);
        if (two) {   // the second part, `rows` rows on
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] -= __bfloat162float(__float2bfloat16_rn(g[j]));
          store_vec<bf16, 8>(static_cast<bf16*>(exps) + static_cast<size_t>(rows) * ld + at, g);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- operands
// Copies a matrix into rows that TMA can read: as it is (PARTS = 1), or fp32
// into PARTS = 3 planes of bfloat16.  A value becomes hi + mid + lo: hi is the value truncated to bfloat16 (so
// that it never overflows), mid and lo round what is left to nearest; the
// rest is below 2^-25 of the value.
// One launch takes x and w where both need it.  `copies` of x serve a w whose
// rows are not on 16-byte boundaries (few_gemm.cu): copy c, its parts c PARTS
// planes on, lies shift(c) columns to the right, with zeros on both sides; or
// the two parts of g.
struct Packing {
  const void* src;
  void* dst;
  long long ld, ld_dst, plane;
  int rows, cols;
  int vectors;              // rows of src take 16-byte loads
  int copies, shift0, step, mask;

  __host__ __device__ long long vecs() const { return copies * rows * (ld_dst / 8); }
};

template <class T, int PARTS, class O>
__global__ void __launch_bounds__(256) loss_pack_kernel(Packing x, Packing w, unsigned* err) {
  grid_launch_dependents();
  grid_dependency_wait();
  const long long all_x = x.vecs(), all = all_x + w.vecs();
  for (long long n = blockIdx.x * 256LL + threadIdx.x; n < all; n += gridDim.x * 256LL) {
    const Packing& m = n < all_x ? x : w;
    const long long i = n < all_x ? n : n - all_x;
    const int per_row = static_cast<int>(m.ld_dst / 8);
    const int line = static_cast<int>(i / per_row);      // at most kFewRows kFewMostClasses, or rows
    const int copy = line / m.rows, r = line - copy * m.rows;
    const int shift = (m.shift0 + copy * m.step) & m.mask;
    const int to = static_cast<int>(i - static_cast<long long>(line) * per_row) * 8, c = to - shift;
    const T* const src = static_cast<const T*>(m.src) + static_cast<size_t>(r) * m.ld;
    const size_t at = static_cast<size_t>(r) * m.ld;
    float v[8];
    if (m.vectors && shift == 0 && c + 8 <= m.cols) {
      if (!GEMM_IN_EXTENT(at + c + 7, stored_extent(m.rows, m.cols, m.ld), err, kSiteBoundsRows)) continue;
      Raw<T, 8> raw;
      raw.load_once(src + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = raw.at(j);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = c + j >= 0 && c + j < m.cols &&
                       GEMM_IN_EXTENT(at + c + j, stored_extent(m.rows, m.cols, m.ld), err, kSiteBoundsRows)
                   ? to_f32(src[c + j])
                   : 0.0f;
    }
    O* const out = static_cast<O*>(m.dst) + copy * PARTS * m.plane + static_cast<size_t>(r) * m.ld_dst + to;
    if constexpr (PARTS == 3) {
      float hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hi[j] = __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u);
        v[j] -= hi[j];
      }
      store_vec<bf16, 8>(out, hi);
#pragma unroll
      for (int part = 1; part < 3; ++part) {
        store_vec<bf16, 8>(out + part * m.plane, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
      }
    } else {
      store_vec<O, 8>(out, v);
    }
  }
}

// ---------------------------------------------------------------- host side
template <class Kernel, class... Args>
int launch(Kernel kernel, dim3 grid, int threads, cudaStream_t stream, int* launches,
           Args... args) {
  if (launch_dependent(kernel, grid, dim3(threads), 0, stream, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  ++*launches;
  return GEMM_F32_OK;
}

struct Call {
  int type;
  int rows, width, vocab;
  const void* x;
  long long ldx;
  const void* w;
  long long ldw;
  const void* targets;
  int target_bits;
  long long ignore;
  int reduction;
  float grad_scale;
  float *loss, *lse, *total;
  void* dx;
  long long lddx;
  void* dw;
  long long lddw;
  size_t piece_bytes;
};

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// Parts of the scratch buffer, handed out in order.
struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += round_up(n, 256);
    return at;
  }
};

// An operand as TMA reads it: where it lies, or copied into scratch because
// its rows are not on 16-byte boundaries, or as three parts of fp32.
struct Operand {
  enum Form { kAsIs, kCopied, kSplit } form = kAsIs;
  size_t at = 0;           // in scratch
  long long ld = 0, plane = 0;
  const void* in(const void* p, const char* scratch) const { return form == kAsIs ? p : scratch + at; }
};

bool on_boundaries(const void* p, long long ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

// `classes`: of a w that x's copies serve, or null.
Operand plan_operand(const void* p, long long ld, int rows, int cols, bool f32, bool split,
                     const FewClasses* classes, Layout& layout) {
  Operand o;
  const int size = f32 ? 4 : 2;
  if (split)
    o.form = Operand::kSplit;
  else if (classes || !on_boundaries(p, ld, size))
    o.form = Operand::kCopied;
  o.ld = ld;
  if (o.form != Operand::kAsIs) {
    o.ld = static_cast<long long>(round_up(static_cast<size_t>(cols) + (classes ? classes->mask : 0), 8));
    o.plane = o.ld * rows;
    o.at = layout.take(static_cast<size_t>(o.plane) * (split ? 6 : size) * (classes ? classes->count : 1));
  }
  return o;
}

Packing packing(const Operand& o, const void* src, long long ld, int rows, int cols, bool f32,
                const FewClasses* classes, char* scratch) {
  Packing m = {src, scratch + o.at, ld, o.ld, o.plane, rows, cols, on_boundaries(src, ld, f32 ? 4 : 2), 1, 0, 0, 0};
  if (classes) {
    m.copies = classes->count;
    m.shift0 = classes->shift0;
    m.step = classes->step;
    m.mask = classes->mask;
  }
  return m;
}

// Packs x and w, which take the same form, or one of them (the other has no rows).
int pack(Operand::Form form, const Packing& x, const Packing& w, bool f32, int num_sms, unsigned* err,
         cudaStream_t stream, int* launches) {
  const long long work = x.vecs() + w.vecs();
  const dim3 grid(static_cast<unsigned>(std::min<long long>((work + 255) / 256, 16LL * num_sms)));
  return form == Operand::kSplit
             ? launch(loss_pack_kernel<float, 3, bf16>, grid, 256, stream, launches, x, w, err)
         : f32 ? launch(loss_pack_kernel<float, 1, float>, grid, 256, stream, launches, x, w, err)
               : launch(loss_pack_kernel<bf16, 1, bf16>, grid, 256, stream, launches, x, w, err);
}

int run(const Call& c, cudaStream_t stream, int* launches, const char** kernel) {
  int device = 0, num_sms = 0;
  unsigned* err = nullptr;
  if (!current_device(&device, &num_sms, &err)) return GEMM_F32_EDEVICE;
  const bool f32 = c.type == GEMM_F32_TYPE_F32, grad = c.dx || c.dw;
  // the losses alone of few rows read a w off 16-byte boundaries where it lies
  // (bfloat16 x 4095 x 65535: 8 rows 114 us against 339 with w copied first,
  // 128 rows 159 against 350); with gradients dx needs the copy anyway
  const FewClasses by_class = few_classes(f32, c.w, c.ldw, c.vocab);
  const bool direct = !grad && !by_class.aligned() && c.rows <= kFewRows && c.vocab >= by_class.count;
  const bool few = direct || c.rows <= (f32 ? kFewRows : kFewRowsBf16);
  *kernel = few ? "few_gemm_kernel" : "half_gemm_kernel";
  const int parts = f32 ? 3 : 1;
  const long long ld_exps = static_cast<long long>(round_up(c.vocab, 256));
  const int piece_bits = few ? kFewPieceBits : kPieceBits;
  const bool two = grad && few && !f32;                // parts of g, one below the other
  const FewClasses twice = {2, 0, 0, 0, 0};            // so x for dw: two copies, not shifted
  const FewClasses* const classes = direct ? &by_class : two && c.dw ? &twice : nullptr;
  const int pieces = direct ? by_class.count * by_class.units
                     : few  ? (c.vocab + kFewPiece - 1) / kFewPiece
                            : static_cast<int>(ld_exps >> kPieceBits);

  // rows per piece: bounded by the exponentials (and the parts of g), or by
  // the statistics alone
  const size_t row_bytes = grad ? static_cast<size_t>(ld_exps) * (f32 ? 4 + 6 : 2)
                                : static_cast<size_t>(pieces) * sizeof(float2);
  const size_t most = grad ? (c.piece_bytes ? c.piece_bytes : kDefaultPieceBytes) : kMostStatsBytes;
  const size_t fit = std::max<size_t>(256, most / row_bytes / 256 * 256);
  const size_t n_pieces = (static_cast<size_t>(c.rows) + fit - 1) / fit;
  const int step = static_cast<int>(std::min<size_t>(
      round_up((static_cast<size_t>(c.rows) + n_pieces - 1) / n_pieces, 256), c.rows));
  const bool sum_dw = c.dw && !f32 && step < c.rows;   // bfloat16 dw of several pieces

  Layout layout;
  const size_t at_arrived = layout.take(sizeof(unsigned));
  const size_t at_factors = layout.take(sizeof(Factors));
  const size_t at_logit = layout.take(sizeof(float) * c.rows);
  const int groups_all = (c.rows - 1) / kJoinRows + 1;
  const size_t at_sums = layout.take(sizeof(float) * groups_all);
  const size_t at_counts = layout.take(sizeof(int) * groups_all);
  const long long ld_stats = static_cast<long long>(round_up(step, 32));
  const size_t at_stats = layout.take(sizeof(float2) * pieces * ld_stats);
  const size_t at_joined = grad ? layout.take(sizeof(float2) * step) : 0;
  const Operand ox = plan_operand(c.x, c.ldx, c.rows, c.width, f32, f32, classes, layout);
  Operand ow;
  ow.ld = c.ldw;
  if (!direct) ow = plan_operand(c.w, c.ldw, c.vocab, c.width, f32, f32 && !few, nullptr, layout);
  size_t at_exps = 0, at_g = 0, at_partials = 0, at_sum = 0;
  if (grad) {
    at_exps = layout.take(static_cast<size_t>(step) * ld_exps * (f32 ? 4 : 2) * (two ? 2 : 1));
    at_g = f32 ? layout.take(static_cast<size_t>(step) * ld_exps * 6) : at_exps;
    size_t partial = 0;
    for (long long r = 0; r < c.rows; r += step) {
      const int n = static_cast<int>(std::min<long long>(step, c.rows - r));
      if (c.dx)
        partial = std::max(partial, few ? few_gemm_scratch(two ? 2 * n : n, c.width, c.vocab, num_sms)
                                        : half_gemm_scratch(n, c.width, c.vocab, parts, num_sms));
      if (c.dw) partial = std::max(partial, half_gemm_scratch(c.vocab, c.width, two ? 2 * n : n, parts, num_sms));
    }
    at_partials = layout.take(partial);
    if (sum_dw) at_sum = layout.take(sizeof(float) * static_cast<size_t>(c.vocab) * c.width);
  }
  char* const scratch = static_cast<char*>(acquire_scratch(device, stream, layout.bytes));
  if (!scratch) return GEMM_F32_ESCRATCH;

  Factors* const factors = reinterpret_cast<Factors*>(scratch + at_factors);
  unsigned* const arrived = reinterpret_cast<unsigned*>(scratch + at_arrived);
  float* const logit = reinterpret_cast<float*>(scratch + at_logit);
  float2* const stats = reinterpret_cast<float2*>(scratch + at_stats);
  const LossTargets all = {c.targets, c.target_bits, c.vocab, c.ignore};
  const Packing px = packing(ox, c.x, c.ldx, c.rows, c.width, f32, classes, scratch);
  const Packing pw = packing(ow, c.w, c.ldw, c.vocab, c.width, f32, nullptr, scratch);
  int rc = GEMM_F32_OK;
  if (ox.form == ow.form && ox.form != Operand::kAsIs) {
    rc = pack(ox.form, px, pw, f32, num_sms, err, stream, launches);
  } else {
    if (ox.form != Operand::kAsIs) rc = pack(ox.form, px, Packing{}, f32, num_sms, err, stream, launches);
    if (rc == GEMM_F32_OK && ow.form != Operand::kAsIs)
      rc = pack(ow.form, Packing{}, pw, f32, num_sms, err, stream, launches);
  }

  const HalfOperand w = {ow.in(c.w, scratch), ow.ld, ow.plane, false};
  for (long long r = 0; rc == GEMM_F32_OK && r < c.rows; r += step) {
    const int n = static_cast<int>(std::min<long long>(step, c.rows - r));
    HalfGemm base = {};
    base.parts = parts;
    base.num_sms = num_sms;
    base.device = device;
    base.err = err;
    const char* const xp = static_cast<const char*>(ox.in(c.x, scratch));
    const HalfOperand x = {xp + static_cast<size_t>(r) * ox.ld * 2, ox.ld, ox.plane, false};
    LossTargets targets = all;
    targets.p = static_cast<const char*>(all.p) + r * (c.target_bits / 8);

    FewGemm few_base = {};
    few_base.f32 = f32;
    few_base.rows = n;
    few_base.width = c.width;
    few_base.vocab = c.vocab;
    few_base.w = w.ptr;
    few_base.ldw = w.ld;
    few_base.num_sms = num_sms;
    few_base.device = device;
    few_base.err = err;
    if (few) {
      FewGemm z = few_base;
      z.b = x;
      z.classes = few_classes(f32, z.w, z.ldw, c.vocab);
      z.stats = stats;
      z.ld_stats = ld_stats;
      z.exps = grad ? scratch + at_exps : nullptr;
      z.ld_exps = ld_exps;
      z.targets = targets;
      z.label_logit = logit;
      z.arrived = arrived;
      rc = launch_few_gemm(z, stream, launches);
    } else {
      HalfGemm z = base;
      z.M = n;
      z.N = c.vocab;
      z.K = c.width;
      z.a = x;
      z.b = w;
      z.stats = stats;
      z.ld_stats = ld_stats;
      z.exps = grad ? scratch + at_exps : nullptr;
      z.ld_exps = ld_exps;
      z.targets = targets;
      z.label_logit = logit + r;
      z.arrived = arrived;
      rc = launch_half_gemm(z, stream, launches);
    }
    if (rc != GEMM_F32_OK) break;
    float2* const joined = grad ? reinterpret_cast<float2*>(scratch + at_joined) : nullptr;
    JoinArgs j = {};
    j.stats = stats;
    j.ld = ld_stats;
    j.pieces = pieces;
    j.rows = n;
    j.targets = targets;
    j.label_logit = logit + r;
    j.loss = c.loss ? c.loss + r : nullptr;
    j.lse = c.lse ? c.lse + r : nullptr;
    j.joined = joined;
    j.all_sums = reinterpret_cast<float*>(scratch + at_sums);
    j.all_counts = reinterpret_cast<int*>(scratch + at_counts);
    j.sums = reinterpret_cast<float*>(scratch + at_sums) + r / kJoinRows;
    j.counts = reinterpret_cast<int*>(scratch + at_counts) + r / kJoinRows;
    j.all_targets = all;
    j.all_rows = c.rows;
    j.first = r == 0;
    j.last = r + step >= c.rows;
    j.mean = c.reduction == GEMM_F32_MEAN;
    j.grad_scale = c.grad_scale;
    j.factors = factors;
    j.total = c.total;
    j.arrived = arrived;
    j.err = err;
    const int join_ctas = (n + kJoinRows - 1) / kJoinRows;
    rc = join_ctas <= num_sms
             ? launch(loss_join_kernel<kJoinThreadsFew>, dim3(join_ctas), kJoinThreadsFew, stream, launches, j)
             : launch(loss_join_kernel<kJoinThreads>, dim3(join_ctas), kJoinThreads, stream, launches, j);
    if (rc != GEMM_F32_OK) break;
    if (!grad) continue;

    // bands of columns: some eight CTAs per SM where the rows alone give fewer
    const int groups = (n + kRescaleRows - 1) / kRescaleRows;
    const int cols = static_cast<int>(round_up(c.vocab, 8));
    const int bands = 8 * num_sms / groups + 1;
    const unsigned band = static_cast<unsigned>(round_up((cols - 1) / bands + 1, kRescaleThreads * 8));
    const dim3 grid(groups, (cols - 1) / band + 1);
    bf16* const gp = reinterpret_cast<bf16*>(scratch + at_g);
    const long long plane = f32 ? static_cast<long long>(step) * ld_exps : 0;
    rc = launch(f32 ? loss_rescale_kernel<3> : loss_rescale_kernel<1>, grid, kRescaleThreads, stream,
                launches, static_cast<const float2*>(stats), ld_stats, piece_bits,
                static_cast<const float2*>(joined), n, cols, band, targets,
                static_cast<void*>(scratch + at_exps), ld_exps, gp, plane, two, err);
    if (rc != GEMM_F32_OK) break;

    base.scale = &factors->grad;
    base.partials = reinterpret_cast<float*>(scratch + at_partials);
    if (c.dx && few) {
      FewGemm d = few_base;
      d.rows = two ? 2 * n : n;
      d.two = two;
      d.b = {gp, ld_exps, plane, false};
      d.dx = c.dx;
      d.lddx = c.lddx;
      d.scale = base.scale;
      d.partials = base.partials;
      rc = launch_few_gemm(d, stream, launches);
      if (rc != GEMM_F32_OK) break;
    } else if (c.dx) {   // dx = s g w: K runs along the vocabulary
      HalfGemm d = base;
      d.M = n;
      d.N = c.width;
      d.K = c.vocab;
      d.a = {gp, ld_exps, plane, false};
      d.b = {w.ptr, w.ld, w.plane, true};
      d.c = static_cast<char*>(c.dx) + static_cast<size_t>(r) * c.lddx * (f32 ? 4 : 2);
      d.ldc = c.lddx;
      d.c_f32 = f32;
      rc = launch_half_gemm(d, stream, launches);
      if (rc != GEMM_F32_OK) break;
    }
    if (c.dw) {   // dw += s g^T x: K runs along the rows
      HalfGemm d = base;
      d.M = c.vocab;
      d.N = c.width;
      d.K = two ? 2 * n : n;
      d.a = {gp, ld_exps, plane, true};
      d.b = {x.ptr, x.ld, x.plane, true};
      const bool last = r + step >= c.rows;
      float* const sum = reinterpret_cast<float*>(scratch + at_sum);
      const bool to_sum = sum_dw && !last;
      d.c = to_sum ? static_cast<void*>(sum) : c.dw;
      d.ldc = to_sum ? c.width : c.lddw;
      d.c_f32 = f32 || to_sum;
      if (r > 0) {
        d.add = sum_dw ? sum : static_cast<const float*>(c.dw);
        d.ldadd = sum_dw ? c.width : c.lddw;
      }
      rc = launch_half_gemm(d, stream, launches);
    }
  }
  return rc;
}

bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

size_t matrix_bytes(int rows, int width, long long ld, size_t size) {
  return (static_cast<size_t>(rows - 1) * ld + width) * size;
}

int checked(Call& c, long long rows, gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (c.type != GEMM_F32_TYPE_F32 && c.type != GEMM_F32_TYPE_BF16) return GEMM_F32_EINVAL;
  if (c.reduction != GEMM_F32_SUM && c.reduction != GEMM_F32_MEAN) return GEMM_F32_EINVAL;
  if (c.target_bits != 32 && c.target_bits != 64) return GEMM_F32_EINVAL;
  if (rows < 0 || rows > INT_MAX || c.width < 1 || c.vocab < 1) return GEMM_F32_EINVAL;
  // tiles and row strides rounded up stay within an int
  if (c.vocab > INT_MAX - 256 || c.width > INT_MAX - 256 || !std::isfinite(c.grad_scale)) return GEMM_F32_EINVAL;
  if (!aligned_to(c.loss, 4) || !aligned_to(c.lse, 4) || !aligned_to(c.total, 4))
    return GEMM_F32_EINVAL;
  const size_t size = c.type == GEMM_F32_TYPE_F32 ? 4 : 2;
  c.rows = static_cast<int>(rows);
  if (!c.w || !aligned_to(c.w, size) || c.ldw < c.width) return GEMM_F32_EINVAL;
  if (c.dw && (!aligned_to(c.dw, size) || c.lddw < c.width)) return GEMM_F32_EINVAL;
  if (rows > 0) {
    if (!c.x || !aligned_to(c.x, size) || c.ldx < c.width) return GEMM_F32_EINVAL;
    if (!c.targets || !aligned_to(c.targets, c.target_bits / 8)) return GEMM_F32_EINVAL;
    if (c.dx && (!aligned_to(c.dx, size) || c.lddx < c.width)) return GEMM_F32_EINVAL;
  }
  const size_t w_bytes = matrix_bytes(c.vocab, c.width, c.ldw, size);
  const size_t x_bytes = rows ? matrix_bytes(c.rows, c.width, c.ldx, size) : 0;
  const size_t dw_bytes = c.dw ? matrix_bytes(c.vocab, c.width, c.lddw, size) : 0;
  const size_t dx_bytes = c.dx && rows ? matrix_bytes(c.rows, c.width, c.lddx, size) : 0;
  if (ranges_overlap(c.dw, dw_bytes, c.w, w_bytes) || ranges_overlap(c.dw, dw_bytes, c.x, x_bytes) ||
      ranges_overlap(c.dx, dx_bytes, c.w, w_bytes) || ranges_overlap(c.dx, dx_bytes, c.x, x_bytes) ||
      ranges_overlap(c.dx, dx_bytes, c.dw, dw_bytes))
    return GEMM_F32_EINVAL;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  if (rows == 0) {   // an empty sum
    int device = 0, num_sms = 0, launches = 0;
    unsigned* err = nullptr;
    if (!c.total && !c.dw) return GEMM_F32_OK;
    if (!current_device(&device, &num_sms, &err)) return GEMM_F32_EDEVICE;
    if (c.total && cudaMemsetAsync(c.total, 0, sizeof(float), stream) != cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    launches += c.total ? 1 : 0;
    if (c.dw) {
      if (cudaMemset2DAsync(c.dw, c.lddw * size, 0, c.width * size, c.vocab, stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return GEMM_F32_ELAUNCH;
      }
      ++launches;
    }
    note_launches(launches, "memset");
    return GEMM_F32_OK;
  }
  int launches = 0;
  const WorkspaceCall call;
  const char* kernel = "none";
  const int rc = run(c, stream, &launches, &kernel);
  if (rc == GEMM_F32_OK) note_launches(launches, kernel);
  return rc;
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" int gemm_f32_vocab_loss(int type, long long rows, int width, int vocab, const void* x,
                                   long long ldx, const void* w, long long ldw, const void* targets,
                                   int target_bits, long long ignore_index, int reduction, float* loss,
                                   float* lse, float* total, gemm_f32_stream_t stream) {
  Call c = {type, 0,    width, vocab, x,       ldx, w, ldw,     targets, target_bits, ignore_index, reduction,
            1.0f, loss, lse,   total, nullptr, 0,   nullptr, 0, 0};
  return checked(c, rows, stream);
}

extern "C" int gemm_f32_vocab_loss_grad(int type, long long rows, int width, int vocab, const void* x,
                                        long long ldx, const void* w, long long ldw,
                                        const void* targets, int target_bits, long long ignore_index,
                                        int reduction, float grad_scale, float* loss, float* lse,
                                        float* total, void* dx, long long lddx, void* dw,
                                        long long lddw, size_t piece_bytes,
                                        gemm_f32_stream_t stream) {
  Call c = {type,       0,    width, vocab, x,  ldx,  w,  ldw,  targets, target_bits, ignore_index, reduction,
            grad_scale, loss, lse,   total, dx, lddx, dw, lddw, piece_bytes};
  return checked(c, rows, stream);
}
