// The norms at a block's ends, with its gate and residual, and their
// gradients (sm_103a).
//
//   p = branch, or its norm;  h = alpha residual + beta gate p;  y = norm(h)
//   hat = (h - mean) rstd, g = dy weight
//   d = dh + rstd (g - sum(g)/D - hat sum(g hat)/D),  dresidual = alpha d
//   e = beta d gate,  dgate = beta d p,  dbranch = e, or through p's norm as d
//
// Bound by memory traffic: each matrix is read or written once, so a row goes
// from its load to its results in the registers of the threads that share it
// (block_rows.cuh), through both norms.  The next rows of all matrices are in
// flight meanwhile, in a ring that bulk copies fill; vectors over the columns
// (weights, a gate per channel) lie in shared memory in the order in which the
// threads hold the columns.  The gradient's grid is persistent: a thread keeps
// its columns and sums their shares of the vectors' gradients in registers; a
// second kernel adds the CTAs' sums in order (no atomics).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gemm_f32_block.h"
#include "block_rows.cuh"
#include "device_common.cuh"
#include "launch.h"
#include "row_common.cuh"
#include "workspace.h"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

constexpr size_t kMostShared = 224 * 1024;   // dynamic; what is static fits beside it
constexpr int kMostStages = 8;

// Vectors over the columns, by their place in VectorArgs.
enum { kWeight, kBias, kPostWeight, kPostBias, kGateVector, kVectors };

struct VectorArgs {
  const void* p[kVectors];               // null where `there`: the default
  int slot[kVectors];                    // of the vectors in shared memory, -1: not there
  int f32;
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
  float* partials;                       // [CTA or cluster][sums][width]
  int sum[kSums];                        // a vector's place in the partials, -1: not wanted
  int sums;
  unsigned* err;
};

__device__ __forceinline__ Pair both(float x) { return pair_of(x, x); }

// What row operators keep in static shared memory.
struct RowShared {
  float part[2][2][kRowWarps];
  float2 ctas[2][kMostCtas];
  uint64_t bars[2];
};

__device__ __forceinline__ RowSums row_sums(RowShared& s, const RowPlan& plan, int group, int rank, unsigned* err) {
  RowSums r = {s.part, s.ctas, smem_addr(s.bars), err, group, plan.lanes, plan.ctas, rank};
  return r;
}

template <class T>
__device__ __forceinline__ bool output_ok(const Output& o, const RowPlan& plan, long long row, unsigned* err) {
  return GEMM_IN_EXTENT(row * o.ld + plan.width - 1, stored_extent(plan.rows, plan.width, o.ld), err,
                        kSiteBoundsRows);
}

// ---------------------------------------------------------------- forward
template <class T, int NE, bool VEC>
__global__ void __launch_bounds__(kAllThreads, 1) block_norm_kernel(const __grid_constant__ BlockArgs a) {
  using Part = RowPart<T, NE, VEC>;
  constexpr int NP = Part::NP;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ RowShared shared;
  const RowPlan& plan = a.plan;
  const int group = threadIdx.x / plan.lanes, t = threadIdx.x % plan.lanes;
  const int rank = plan.ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool producer = group == plan.groups;
  const RingPlace ring(plan, smem_rows, rank);
  RowSums sums = row_sums(shared, plan, group, rank, a.err);
  if (threadIdx.x == 0) {
    if (plan.ctas > 1)
      for (int i = 0; i < 2; ++i) mbar_init(sums.bars + 8u * i, 1);
    ring.init(plan);
  }
  __syncthreads();
  if (plan.ctas > 1) cluster_sync();     // every CTA of the cluster runs
  grid_launch_dependents();
  grid_dependency_wait();
  float* const columns = reinterpret_cast<float*>(smem_rows);
  const int slots = Part::slots(plan.lanes);
#pragma unroll 1
  for (int v = 0; v < kVectors; ++v)
    if (a.vectors.slot[v] >= 0)
      fill_columns<T, Part>(columns + a.vectors.slot[v] * slots, a.vectors.p[v], a.vectors.f32,
                            v == kWeight || v == kPostWeight ? 1.0f : 0.0f, plan.lanes, ring.col0, ring.width);
  __syncthreads();
  const Part mine(t, plan.lanes, ring.width);
  const float inv = 1.0f / static_cast<float>(plan.width);
  auto vector = [&](int v, Pair(&w)[NP]) { mine.load_columns(columns + a.vectors.slot[v] * slots, w); };

  // x around its mean (0 for rms), 1 / its root mean square there.
  auto normalise = [&](Pair(&x)[NP], float& mean, float& rstd) {
    float s[1];
    mean = 0.0f;
    if (!a.rms) {
      Pair sum = 0;
#pragma unroll
      for (int j = 0; j < NP; ++j) sum = add2(sum, x[j]);
      s[0] = sum_of(sum);
      sums.add<1>(s);
      mean = s[0] * inv;
#pragma unroll
      for (int j = 0; j < NP; ++j) x[j] = add2(x[j], both(-mean));
      mine.drop(x);
    }
    Pair sum = 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) sum = fma2(x[j], x[j], sum);
    s[0] = sum_of(sum);
    sums.add<1>(s);
    rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
  };

  if (producer) produce_rows(a.in, plan, ring, a.err);
  RingReader reader = {ring, plan, a.err, group};
  for (long long row = ring.first * plan.groups + group; !producer && row < plan.rows; row += ring.step * plan.groups) {
    reader.wait();
    Pair p[NP], x[NP], w[NP];
    mine.load(reader.at(a.in[kInBranch], row, VEC), p);
    mine.load(reader.at(a.in[kInResidual], row, VEC), x);
    Pair gate[NP];
    if (a.gate == kElementGate) mine.load(reader.at(a.in[kInGate], row, VEC), gate);
    reader.release();
    float mean, rstd, mean_b = 0.0f, rstd_b = 0.0f;
    if (a.post) {
      normalise(p, mean_b, rstd_b);
      vector(kPostWeight, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) p[j] = mul2(mul2(p[j], both(rstd_b)), w[j]);
      if (a.vectors.slot[kPostBias] >= 0) {
        vector(kPostBias, w);
#pragma unroll
        for (int j = 0; j < NP; ++j) p[j] = add2(p[j], w[j]);
      }
    }
    if (a.gate == kChannelGate) vector(kGateVector, gate);
    if (a.gate != kNoGate) {
#pragma unroll
      for (int j = 0; j < NP; ++j) p[j] = mul2(p[j], gate[j]);
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) x[j] = fma2(p[j], both(a.beta), mul2(x[j], both(a.alpha)));
    if (a.h.p && output_ok<T>(a.h, plan, row, a.err)) {
      // an h that is an input: all of this row has been read
      mine.store(static_cast<T*>(a.h.p) + row * a.h.ld + ring.col0, x);
    }
    normalise(x, mean, rstd);
    vector(kWeight, w);
#pragma unroll
    for (int j = 0; j < NP; ++j) x[j] = mul2(mul2(x[j], both(rstd)), w[j]);
    if (a.vectors.slot[kBias] >= 0) {
      vector(kBias, w);
#pragma unroll
      for (int j = 0; j < NP; ++j) x[j] = add2(x[j], w[j]);
    }
    if (output_ok<T>(a.y, plan, row, a.err)) mine.store(static_cast<T*>(a.y.p) + row * a.y.ld + ring.col0, x);
    if (t == 0 && rank == 0 && a.stats) {
      a.stats[row] = mean;
      a.stats[plan.rows + row] = rstd;
      if (a.post) {
        a.stats[2 * plan.rows + row] = mean_b;
        a.stats[3 * plan.rows + row] = rstd_b;
      }
    }
  }
  if (plan.ctas > 1) cluster_sync();     // no CTA leaves while another may write to it
}

// ---------------------------------------------------------------- gradient
template <class T, bool VEC>
__global__ void __launch_bounds__(kAllThreads, 1) block_norm_grad_kernel(const __grid_constant__ BlockGradArgs a) {
  constexpr int NE = 8;
  using Part = RowPart<T, NE, VEC>;
  constexpr int NP = Part::NP;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ RowShared shared;
  const RowPlan& plan = a.plan;
  const int group = threadIdx.x / plan.lanes, t = threadIdx.x % plan.lanes;
  const int rank = plan.ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool producer = group == plan.groups;
  const RingPlace ring(plan, smem_rows, rank);
  RowSums sums = row_sums(shared, plan, group, rank, a.err);
  if (threadIdx.x == 0) {
    if (plan.ctas > 1)
      for (int i = 0; i < 2; ++i) mbar_init(sums.bars + 8u * i, 1);
    ring.init(plan);
  }
  __syncthreads();
  if (plan.ctas > 1) cluster_sync();     // every CTA of the cluster runs
  grid_launch_dependents();
  grid_dependency_wait();
  float* const columns = reinterpret_cast<float*>(smem_rows);
  const int slots = Part::slots(plan.lanes);
#pragma unroll 1
  for (int v = 0; v < kVectors; ++v)
    if (a.vectors.slot[v] >= 0)
      fill_columns<T, Part>(columns + a.vectors.slot[v] * slots, a.vectors.p[v], a.vectors.f32,
                            v == kWeight || v == kPostWeight ? 1.0f : 0.0f, plan.lanes, ring.col0, ring.width);
  __syncthreads();
  const Part mine(t, plan.lanes, ring.width);
  const float inv = 1.0f / static_cast<float>(plan.width);
  auto vector = [&](int v, Pair(&w)[NP]) { mine.load_columns(columns + a.vectors.slot[v] * slots, w); };
  Pair total[kSums][NP];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int j = 0; j < NP; ++j) total[k][j] = 0;

  float stat[4] = {0.0f, 0.0f, 0.0f, 0.0f};      // this row's, loaded under the row before
  auto load_stats = [&](long long r) {
    if (r >= plan.rows) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < 2 || a.post) stat[k] = __ldg(a.stats + k * plan.rows + r);
  };
  if (producer) produce_rows(a.in, plan, ring, a.err);
  RingReader reader = {ring, plan, a.err, group};
  const long long step = ring.step * plan.groups;
  long long row = producer ? plan.rows : ring.first * plan.groups + group;
  load_stats(row);
  for (; row < plan.rows; row += step) {
    reader.wait();
    const float mean = a.rms ? 0.0f : stat[0], rstd = stat[1];
    const float mean_b = a.rms ? 0.0f : stat[2], rstd_b = stat[3];
    load_stats(row + step);
    // all of the row into registers, so that its stage is free
    Pair c[NP], g[NP], d[NP], b[NP], gate[NP], w[NP];
    if (a.in[kGradHExponents].p)
      mine.load_saved(reader.at(a.in[kGradH], row, true), reader.at(a.in[kGradHExponents], row, true), c);
    else
      mine.load(reader.at(a.in[kGradH], row, VEC), c);
    mine.load(reader.at(a.in[kGradDy], row, VEC), g);
    if (a.in[kGradDh].p) {
      mine.load(reader.at(a.in[kGradDh], row, VEC), d);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) d[j] = 0;
    }
    if (a.branch) {
      if (a.in[kGradBranchExponents].p)
        mine.load_saved(reader.at(a.in[kGradBranch], row, true), reader.at(a.in[kGradBranchExponents], row, true), b);
      else
        mine.load(reader.at(a.in[kGradBranch], row, VEC), b);
    }
    if (a.gate == kElementGate) mine.load(reader.at(a.in[kGradGate], row, VEC), gate);
    reader.release();
    // c = h - mean in place of hat = c rstd: where rstd is 0 (squares that
    // overflowed) or c is, hat is 0 and never 0 times infinity
    vector(kWeight, w);
    Pair sg = 0, sgc = 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      c[j] = add2(c[j], both(-mean));
      total[kSumWeight][j] = fma2(mul2(g[j], both(rstd)), c[j], total[kSumWeight][j]);
      total[kSumBias][j] = add2(total[kSumBias][j], g[j]);
      g[j] = mul2(g[j], w[j]);
      sg = add2(sg, g[j]);
      sgc = fma2(g[j], c[j], sgc);
    }
    float s[2] = {sum_of(sg), rstd != 0.0f ? sum_of(sgc) * rstd : 0.0f};
    sums.add<2>(s);
    {
      const float c1 = a.rms ? 0.0f : -s[0] * inv, c2 = -s[1] * inv * rstd;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        d[j] = fma2(fma2(c[j], both(c2), add2(g[j], both(c1))), both(rstd), d[j]);
    }
    if (a.dresidual.p && output_ok<T>(a.dresidual, plan, row, a.err)) {
#pragma unroll
      for (int j = 0; j < NP; ++j) g[j] = mul2(d[j], both(a.alpha));
      mine.store(static_cast<T*>(a.dresidual.p) + row * a.dresidual.ld + ring.col0, g);
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) d[j] = mul2(d[j], both(a.beta));
    if (a.branch) {
      mine.drop(d);
      if (a.post) {
#pragma unroll
        for (int j = 0; j < NP; ++j) b[j] = add2(b[j], both(-mean_b));
      }
      if (a.gate != kNoGate) {
        Pair p[NP];
        if (a.post) {
          vector(kPostWeight, w);
#pragma unroll
          for (int j = 0; j < NP; ++j) p[j] = mul2(mul2(b[j], both(rstd_b)), w[j]);
          if (a.vectors.slot[kPostBias] >= 0) {
            vector(kPostBias, w);
#pragma unroll
            for (int j = 0; j < NP; ++j) p[j] = add2(p[j], w[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NP; ++j) p[j] = b[j];
        }
        if (a.gate == kChannelGate) {
          vector(kGateVector, gate);
#pragma unroll
          for (int j = 0; j < NP; ++j) total[kSumGate][j] = fma2(d[j], p[j], total[kSumGate][j]);
        } else if (a.dgate.p && output_ok<T>(a.dgate, plan, row, a.err)) {
#pragma unroll
          for (int j = 0; j < NP; ++j) p[j] = mul2(d[j], p[j]);
          mine.store(static_cast<T*>(a.dgate.p) + row * a.dgate.ld + ring.col0, p);
        }
#pragma unroll
        for (int j = 0; j < NP; ++j) d[j] = mul2(d[j], gate[j]);
      }
      if (a.post) {
        vector(kPostWeight, w);
        Pair se = 0, seb = 0;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          total[kSumPostWeight][j] = fma2(mul2(d[j], both(rstd_b)), b[j], total[kSumPostWeight][j]);
          total[kSumPostBias][j] = add2(total[kSumPostBias][j], d[j]);
          d[j] = mul2(d[j], w[j]);
          se = add2(se, d[j]);
          seb = fma2(d[j], b[j], seb);
        }
        s[0] = sum_of(se);
        s[1] = rstd_b != 0.0f ? sum_of(seb) * rstd_b : 0.0f;
        sums.add<2>(s);
        const float c1 = a.rms ? 0.0f : -s[0] * inv, c2 = -s[1] * inv * rstd_b;
#pragma unroll
        for (int j = 0; j < NP; ++j) d[j] = mul2(fma2(b[j], both(c2), add2(d[j], both(c1))), both(rstd_b));
      }
    }
    if (a.dbranch.p && output_ok<T>(a.dbranch, plan, row, a.err))
      mine.store(static_cast<T*>(a.dbranch.p) + row * a.dbranch.ld + ring.col0, d);
  }
  if (plan.ctas > 1) cluster_sync();     // no CTA leaves while another may write to it
  if (!a.sums) return;
  // the groups' sums, added in group order: one row of partials per CTA (or
  // cluster) and vector; what was the ring makes room
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    if (a.sum[k] < 0) continue;
    __syncthreads();
    float* const own = columns + group * slots;
#pragma unroll
    for (int q = 0; q < (producer ? 0 : NE / 4); ++q) {
      float4 f;
      unpair(total[k][2 * q], f.x, f.y);
      unpair(total[k][2 * q + 1], f.z, f.w);
      *reinterpret_cast<float4*>(mine.quad(own, q)) = f;
    }
    __syncthreads();
    float* const to = a.partials +
                      (static_cast<size_t>(blockIdx.x / plan.ctas) * a.sums + a.sum[k]) * plan.width + ring.col0;
    for (int slot = threadIdx.x; slot < slots; slot += blockDim.x) {
      const int c = Part::column_of_slot(slot, plan.lanes);
      if (c >= ring.width) continue;
      float v = columns[slot];
      for (int i = 1; i < plan.groups; ++i) v += columns[i * slots + slot];
      to[c] = v;
    }
  }
}

// ---------------------------------------------------------------- rows wider than the ring's
// A CTA per row that reads its matrices again for each of the row's sums.
constexpr int kWideThreads = 512;

template <class T>
__device__ __forceinline__ float element(const RowSource& m, long long row, int d) {
  return to_f32(reinterpret_cast<const T*>(m.p + row * m.ld)[d]);
}
template <class T>
__device__ __forceinline__ float element(const RowSource& m, const RowSource& exponents, long long row, int d) {
  if (!exponents.p) return element<T>(m, row, d);
  const uint32_t code = reinterpret_cast<const uint8_t*>(m.p + row * m.ld)[d];
  return values_of(code).x *
         power_of(reinterpret_cast<const uint8_t*>(exponents.p + row * exponents.ld)[d / kSavedBlock]);
}

// Value d of a vector.
template <class T>
__device__ __forceinline__ float vector_at(const VectorArgs& a, int v, int d) {
  if (a.slot[v] < 0) return 0.0f;
  if (!a.p[v]) return v == kWeight || v == kPostWeight ? 1.0f : 0.0f;
  return a.f32 ? __ldg(static_cast<const float*>(a.p[v]) + d) : to_f32(static_cast<const T*>(a.p[v])[d]);
}

template <int N>
__device__ __forceinline__ void wide_sum(float (&v)[N], float (&part)[2][kWideThreads / 32]) {
  warp_sum<N>(v);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[i][warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = part[i][lane & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

template <class T>
__global__ void __launch_bounds__(kWideThreads) block_norm_wide_kernel(const __grid_constant__ BlockArgs a) {
  __shared__ float part[2][kWideThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int width = a.plan.width;
  const float inv = 1.0f / static_cast<float>(width);
  for (long long row = blockIdx.x; row < a.plan.rows; row += gridDim.x) {
    auto statistics = [&](auto value, float& mean, float& rstd) {
      float s[1] = {0.0f};
      mean = 0.0f;
      if (!a.rms) {
        for (int d = threadIdx.x; d < width; d += kWideThreads) s[0] += value(d);
        wide_sum<1>(s, part);
        mean = s[0] * inv;
        s[0] = 0.0f;
      }
      for (int d = threadIdx.x; d < width; d += kWideThreads) {
        const float x = value(d) - mean;
        s[0] = fmaf(x, x, s[0]);
      }
      wide_sum<1>(s, part);
      rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    };
    float mean, rstd, mean_b = 0.0f, rstd_b = 0.0f;
    if (a.post) statistics([&](int d) { return element<T>(a.in[kInBranch], row, d); }, mean_b, rstd_b);
    auto h = [&](int d) {
      float p = element<T>(a.in[kInBranch], row, d);
      if (a.post)
        p = (p - mean_b) * rstd_b * vector_at<T>(a.vectors, kPostWeight, d) + vector_at<T>(a.vectors, kPostBias, d);
      if (a.gate == kChannelGate) p *= vector_at<T>(a.vectors, kGateVector, d);
      if (a.gate == kElementGate) p *= element<T>(a.in[kInGate], row, d);
      return fmaf(p, a.beta, element<T>(a.in[kInResidual], row, d) * a.alpha);
    };
    statistics(h, mean, rstd);
    // an output that is an input: each thread reads its elements before it writes them
    for (int d = threadIdx.x; d < width; d += kWideThreads) {
      const float x = h(d);
      if (a.h.p && output_ok<T>(a.h, a.plan, row, a.err))
        static_cast<T*>(a.h.p)[row * a.h.ld + d] = from_f32<T>(x);
      if (output_ok<T>(a.y, a.plan, row, a.err))
        static_cast<T*>(a.y.p)[row * a.y.ld + d] = from_f32<T>(
            (x - mean) * rstd * vector_at<T>(a.vectors, kWeight, d) + vector_at<T>(a.vectors, kBias, d));
    }
    if (threadIdx.x == 0 && a.stats) {
      a.stats[row] = mean;
      a.stats[a.plan.rows + row] = rstd;
      if (a.post) {
        a.stats[2 * a.plan.rows + row] = mean_b;
        a.stats[3 * a.plan.rows + row] = rstd_b;
      }
    }
  }
}

// The vectors' gradients are summed in the CTA's own partials.
template <class T>
__global__ void __launch_bounds__(kWideThreads) block_norm_grad_wide_kernel(const __grid_constant__ BlockGradArgs a) {
  __shared__ float part[2][kWideThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int width = a.plan.width;
  const float inv = 1.0f / static_cast<float>(width);
  for (long long row = blockIdx.x; row < a.plan.rows; row += gridDim.x) {
    const float mean = a.rms ? 0.0f : a.stats[row], rstd = a.stats[a.plan.rows + row];
    const float mean_b = a.post && !a.rms ? a.stats[2 * a.plan.rows + row] : 0.0f;
    const float rstd_b = a.post ? a.stats[3 * a.plan.rows + row] : 0.0f;
    auto centred = [&](int d) { return element<T>(a.in[kGradH], a.in[kGradHExponents], row, d) - mean; };
    auto branch = [&](int d) { return element<T>(a.in[kGradBranch], a.in[kGradBranchExponents], row, d) - mean_b; };
    auto normed = [&](int d) { return element<T>(a.in[kGradDy], row, d) * vector_at<T>(a.vectors, kWeight, d); };
    auto gate = [&](int d) {
      return a.gate == kChannelGate   ? vector_at<T>(a.vectors, kGateVector, d)
             : a.gate == kElementGate ? element<T>(a.in[kGradGate], row, d)
                                      : 1.0f;
    };
    float s[2] = {0.0f, 0.0f};
    for (int d = threadIdx.x; d < width; d += kWideThreads) {
      const float g = normed(d);
      s[0] += g;
      s[1] = fmaf(g, centred(d), s[1]);
    }
    s[1] = rstd != 0.0f ? s[1] * rstd : 0.0f;
    wide_sum<2>(s, part);
    const float c1 = a.rms ? 0.0f : -s[0] * inv, c2 = -s[1] * inv * rstd;
    auto through = [&](int d) {
      const float dh = a.in[kGradDh].p ? element<T>(a.in[kGradDh], row, d) : 0.0f;
      return fmaf(fmaf(centred(d), c2, normed(d) + c1), rstd, dh);
    };
    float c3 = 0.0f, c4 = 0.0f;
    if (a.post) {
      s[0] = s[1] = 0.0f;
      for (int d = threadIdx.x; d < width; d += kWideThreads) {
        const float e = through(d) * a.beta * gate(d) * vector_at<T>(a.vectors, kPostWeight, d);
        s[0] += e;
        s[1] = fmaf(e, branch(d), s[1]);
      }
      s[1] = rstd_b != 0.0f ? s[1] * rstd_b : 0.0f;
      wide_sum<2>(s, part);
      c3 = a.rms ? 0.0f : -s[0] * inv;
      c4 = -s[1] * inv * rstd_b;
    }
    // an output that is an input: each thread reads its elements before it writes them
    for (int d = threadIdx.x; d < width; d += kWideThreads) {
      const float dy = element<T>(a.in[kGradDy], row, d), c = centred(d), dd = through(d);
      const float e = dd * a.beta;
      const float b = a.branch ? branch(d) : 0.0f, by = gate(d), pw = vector_at<T>(a.vectors, kPostWeight, d);
      const float p = a.post ? b * rstd_b * pw + vector_at<T>(a.vectors, kPostBias, d) : b;
      auto add = [&](int k, float v) {
        if (a.sum[k] < 0) return;
        float* const to = a.partials + (static_cast<size_t>(blockIdx.x) * a.sums + a.sum[k]) * width + d;
        *to = row == blockIdx.x ? v : *to + v;
      };
      add(kSumWeight, dy * rstd * c);
      add(kSumBias, dy);
      if (a.gate == kChannelGate) add(kSumGate, e * p);
      add(kSumPostWeight, e * by * rstd_b * b);
      add(kSumPostBias, e * by);
      if (a.dresidual.p && output_ok<T>(a.dresidual, a.plan, row, a.err))
        static_cast<T*>(a.dresidual.p)[row * a.dresidual.ld + d] = from_f32<T>(dd * a.alpha);
      if (a.dgate.p && a.gate == kElementGate && output_ok<T>(a.dgate, a.plan, row, a.err))
        static_cast<T*>(a.dgate.p)[row * a.dgate.ld + d] = from_f32<T>(e * p);
      const float db = a.post ? rstd_b * fmaf(b, c4, e * by * pw + c3) : e * by;
      if (a.dbranch.p && output_ok<T>(a.dbranch, a.plan, row, a.err))
        static_cast<T*>(a.dbranch.p)[row * a.dbranch.ld + d] = from_f32<T>(db);
    }
  }
}

// ---------------------------------------------------------------- vectors' gradients
// Partial sums of 32 columns of one vector per CTA, added in CTA order: 32
// chains of every 32nd CTA, then the chains in order.
struct ColumnArgs {
  const float* partials;
  void* out[kSums];                      // by their place in the partials
  int sums, ctas, width;
};

template <class WT>
__global__ void __launch_bounds__(1024) block_columns_kernel(const ColumnArgs a) {
  __shared__ float chains[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, chain = threadIdx.x >> 5;
  const int k = blockIdx.y;
  const long long d = blockIdx.x * 32LL + lane;
  float v = 0.0f;
  if (d < a.width)
    for (int c = chain; c < a.ctas; c += 32) v += __ldcg(a.partials + (static_cast<size_t>(c) * a.sums + k) * a.width + d);
  chains[chain][lane] = v;
  __syncthreads();
  float s[1] = {chains[lane][chain]};    // lane: the chain
  warp_sum<1>(s);
  const long long to = blockIdx.x * 32LL + chain;
  if (lane == 0 && to < a.width) static_cast<WT*>(a.out[k])[to] = from_f32<WT>(s[0]);
}

// ---------------------------------------------------------------- host side
size_t type_size(int type) { return type == GEMM_F32_TYPE_F32 ? 4 : 2; }

bool aligned_to(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool matrix_ok(const void* p, long long ld, int width, size_t size) { return p && aligned_to(p, size) && ld >= width; }

size_t matrix_bytes(long long rows, int width, long long ld, size_t size) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * ld + width) * size : 0;
}

// An element's address within its matrix fits in 63 bits.
bool addressable(long long rows, long long ld) { return rows == 0 || ld <= LLONG_MAX / 8 / rows; }

struct Matrix {
  const void* p;
  long long ld;
};

RowSource source(const void* p, long long ld, int size, const RowPlan& plan) {
  RowSource m = {};
  if (!p) return m;
  m.p = static_cast<const char*>(p);
  m.ld = ld * size;
  m.size = size;
  m.end = m.p + matrix_bytes(plan.rows, plan.width, ld, size);
  return m;
}

// Bytes of 8-bit rows, all of which may be read.
RowSource saved_source(const void* p, long long ld, bool exponents, const RowPlan& plan) {
  RowSource m = {};
  if (!p) return m;
  m.p = static_cast<const char*>(p);
  m.ld = ld;
  m.size = exponents ? 0 : 1;
  m.end = m.p + plan.rows * ld;
  return m;
}

// Whether rows start on 16-byte boundaries and hold whole vectors.
bool vector_rows(const void* p, long long ld, int width, size_t size) {
  return aligned_to(p, 16) && ld * size % 16 == 0 && width * size % 16 == 0;
}

// Lays out the rows of `in` over lanes of `ne` elements, groups and ring;
// false where a row is too wide.
bool plan_rows(RowPlan& plan, RowSource* in, int n, int vectors, int ne, bool aligned, int num_sms, size_t* bytes,
               int* grid) {
  for (int ctas = 1; ctas <= kMostCtas; ctas *= 2) {
    if (ctas > num_sms) return false;
    const int slice = ctas == 1 ? plan.width : ((plan.width - 1) / ctas / kSliceUnit + 1) * kSliceUnit;
    if (slice > kRowThreads * ne) continue;
    plan.ctas = ctas;
    plan.slice = slice;
    plan.lanes = 32 * ((slice - 1) / (32 * ne) + 1);
    const long long units = num_sms / ctas;
    plan.groups = static_cast<int>(std::min<long long>(ctas > 1 ? 1 : kRowThreads / plan.lanes,
                                                       (plan.rows - 1) / units + 1));
    const size_t columns = static_cast<size_t>(vectors) * ne * plan.lanes * sizeof(float);
    size_t stage = 0, stages = 0;
    for (;; --plan.groups) {             // two chunks in flight, or fewer groups
      stage = 0;
      for (int i = 0; i < n; ++i) {
        if (!in[i].p) continue;
        const size_t row = source_bytes(in[i].size, slice);
        in[i].packed = ctas == 1 && in[i].ld == static_cast<long long>(row);
        in[i].pitch = static_cast<uint32_t>(in[i].packed ? row : (row + 15) / 16 * 16 + (aligned || in[i].size < 2 ? 0 : 16));
        in[i].at = static_cast<uint32_t>(stage);
        stage += (static_cast<size_t>(plan.groups) * in[i].pitch + 15) / 16 * 16 + (in[i].packed && !aligned ? 16 : 0);
      }
      stages = columns < kMostShared ? (kMostShared - columns) / (stage + 16) : 0;
      if (stages >= 2 || plan.groups == 1) break;
    }
    if (stages < 2) continue;
    plan.stage_bytes = static_cast<uint32_t>(stage);
    plan.ring_at = static_cast<uint32_t>(columns);
    plan.stages = static_cast<int>(std::min<size_t>(stages, kMostStages));
    const long long need = (plan.rows - 1) / plan.groups + 1;
    *grid = static_cast<int>(std::min<long long>(units, need)) * ctas;
    // the groups' sums take the place of the ring
    *bytes = std::max(columns + static_cast<size_t>(plan.stages) * (stage + 16),
                      static_cast<size_t>(plan.groups) * ne * plan.lanes * sizeof(float));
    return true;
  }
  return false;
}

constexpr int kMaxDevices = 64;

// Sets a kernel's shared memory up, once per device, and launches it; where
// CTAs form clusters, with no more of them than run at once (`grid` is
// reduced to that).
template <auto Kernel, class Args>
int launch_rows(const Args& a, int device, int* grid, size_t bytes, cudaStream_t stream) {
  static std::atomic<int> clusters[kMaxDevices][4];   // at a time, per log2 of their CTAs; 1 for single CTAs
  const RowPlan& plan = a.plan;
  std::atomic<int>& kept = clusters[device % kMaxDevices][plan.ctas == 1 ? 0 : plan.ctas == 2 ? 1 : plan.ctas == 4 ? 2 : 3];
  int most = kept.load();
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(*grid);
  config.blockDim = dim3(plan.groups * plan.lanes + 32);
  config.dynamicSmemBytes = bytes;
  config.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = plan.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  if (most == 0) {
    most = 1;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostShared)) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    if (plan.ctas > 1) {
      cudaLaunchConfig_t full = config;
      full.gridDim = dim3(512 / plan.ctas * plan.ctas);
      full.blockDim = dim3(kAllThreads);
      full.dynamicSmemBytes = kMostShared;
      full.attrs = attr + 1;
      full.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&most, Kernel, &full) != cudaSuccess || most < 1) {
        (void)cudaGetLastError();
        return GEMM_F32_ELAUNCH;
      }
    }
    kept.store(most);
  }
  if (plan.ctas > 1) {
    *grid = std::min(*grid, most * plan.ctas);
    config.gridDim = dim3(*grid);
  }
  config.attrs = attr;
  config.numAttrs = plan.ctas > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&config, Kernel, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

template <class Kernel, class Args>
int launch_plain(Kernel kernel, dim3 grid, int threads, cudaStream_t stream, const Args& a) {
  if (launch_dependent(kernel, grid, dim3(threads), 0, stream, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

template <class T>
int forward(BlockArgs& a, int vectors, bool aligned, int device, int num_sms, cudaStream_t stream, const char** kernel) {
  size_t bytes = 0;
  int grid = 0;
  *kernel = "block_norm_kernel";
  const bool wide_threads = a.plan.width > kRowThreads * 8;
  const int ne = wide_threads ? 16 : 8;
  if (!plan_rows(a.plan, a.in, kInputs, vectors, ne, aligned, num_sms, &bytes, &grid)) {
    *kernel = "block_norm_wide_kernel";
    return launch_plain(block_norm_wide_kernel<T>, dim3(static_cast<unsigned>(std::min<long long>(a.plan.rows, 4LL * num_sms))),
                        kWideThreads, stream, a);
  }
  if (ne == 8)
    return aligned ? launch_rows<block_norm_kernel<T, 8, true>>(a, device, &grid, bytes, stream)
                   : launch_rows<block_norm_kernel<T, 8, false>>(a, device, &grid, bytes, stream);
  return aligned ? launch_rows<block_norm_kernel<T, 16, true>>(a, device, &grid, bytes, stream)
                 : launch_rows<block_norm_kernel<T, 16, false>>(a, device, &grid, bytes, stream);
}

template <class T>
int gradient(BlockGradArgs& a, void* const (&vectors_out)[kSums], int vectors, bool aligned, int weight_type, int device,
             int num_sms, cudaStream_t stream, int* launches, const char** kernel) {
  ColumnArgs c = {};
  c.width = a.plan.width;
  for (int k = 0; k < kSums; ++k) {
    a.sum[k] = vectors_out[k] ? a.sums++ : -1;
    if (vectors_out[k]) c.out[a.sum[k]] = vectors_out[k];
  }
  int rc = GEMM_F32_OK;
  *kernel = "block_columns_kernel";
  if (a.plan.rows > 0) {
    size_t bytes = 0;
    int grid = 0;
    const bool ring = plan_rows(a.plan, a.in, kGradInputs, vectors, 8, aligned, num_sms, &bytes, &grid);
    const int bands = ring ? grid / a.plan.ctas : static_cast<int>(std::min<long long>(a.plan.rows, 2LL * num_sms));
    if (a.sums) {
      a.partials = static_cast<float*>(acquire_scratch(
          device, stream, sizeof(float) * static_cast<size_t>(bands) * a.sums * a.plan.width));
      if (!a.partials) return GEMM_F32_ESCRATCH;
    }
    if (ring) {
      *kernel = "block_norm_grad_kernel";
      rc = aligned ? launch_rows<block_norm_grad_kernel<T, true>>(a, device, &grid, bytes, stream)
                   : launch_rows<block_norm_grad_kernel<T, false>>(a, device, &grid, bytes, stream);
      c.ctas = grid / a.plan.ctas;
    } else {
      *kernel = "block_norm_grad_wide_kernel";
      rc = launch_plain(block_norm_grad_wide_kernel<T>, dim3(bands), kWideThreads, stream, a);
      c.ctas = bands;
    }
    ++*launches;
  }
  if (rc == GEMM_F32_OK && a.sums) {
    c.partials = a.partials;
    c.sums = a.sums;
    const dim3 blocks(static_cast<unsigned>((c.width + 31LL) / 32), a.sums);
    rc = weight_type == GEMM_F32_TYPE_F32 ? launch_plain(block_columns_kernel<float>, blocks, 1024, stream, c)
                                          : launch_plain(block_columns_kernel<bf16>, blocks, 1024, stream, c);
    ++*launches;
  }
  return rc;
}

// What both entry points ask of the block's description.
bool block_ok(const gemm_f32_block_t* b) {
  if (!b) return false;
  if (b->type != GEMM_F32_TYPE_F32 && b->type != GEMM_F32_TYPE_BF16) return false;
  if (b->weight_type != GEMM_F32_TYPE_F32 && b->weight_type != b->type) return false;
  if (b->norm != GEMM_F32_NORM_LAYER && b->norm != GEMM_F32_NORM_RMS) return false;
  if ((b->post != 0 && b->post != 1) || b->rows < 0 || b->width < 1) return false;
  if (!std::isfinite(b->residual_scale) || !std::isfinite(b->branch_scale)) return false;
  if (b->norm == GEMM_F32_NORM_RMS && (b->bias || b->post_bias)) return false;
  if (!b->post && (b->post_weight || b->post_bias)) return false;
  const size_t es = type_size(b->type), ws = type_size(b->weight_type);
  if (!aligned_to(b->weight, ws) || !aligned_to(b->bias, ws) || !aligned_to(b->post_weight, ws) ||
      !aligned_to(b->post_bias, ws))
    return false;
  if (b->gate) {
    if (b->ld_gate == 0) return aligned_to(b->gate, ws);
    return matrix_ok(b->gate, b->ld_gate, b->width, es) && addressable(b->rows, b->ld_gate);
  }
  return true;
}

int gate_of(const gemm_f32_block_t& b) { return !b.gate ? kNoGate : b.ld_gate == 0 ? kChannelGate : kElementGate; }

// The vectors that the kernels keep; returns how many.
int vectors_of(const gemm_f32_block_t& b, bool forward, VectorArgs& v) {
  const void* const p[kVectors] = {b.weight, b.bias, b.post_weight, b.post_bias, b.gate};
  const int gate = gate_of(b);
  // the bias of the norm of h does not enter its gradient, that of the
  // branch's norm only through the gate's
  const bool there[kVectors] = {true, forward && b.bias, b.post != 0, b.post_bias && (forward || gate != kNoGate),
                                gate == kChannelGate};
  int n = 0;
  for (int i = 0; i < kVectors; ++i) {
    v.p[i] = there[i] ? p[i] : nullptr;
    v.slot[i] = there[i] ? n++ : -1;
  }
  v.f32 = b.weight_type == GEMM_F32_TYPE_F32;
  return n;
}

// An output that is one of the matrices itself, with the same stride, or
// apart from all of them; and apart from `others`, further outputs, and from
// 8-bit rows.
bool output_fits(const Matrix& out, const Matrix* in, int n_in, const Matrix* others, int n_others, long long rows,
                 int width, size_t size) {
  const size_t bytes = matrix_bytes(rows, width, out.ld, size);
  for (int i = 0; i < n_in; ++i) {
    if (!in[i].p || (out.p == in[i].p && out.ld == in[i].ld)) continue;
    if (ranges_overlap(out.p, bytes, in[i].p, matrix_bytes(rows, width, in[i].ld, size))) return false;
  }
  for (int i = 0; i < n_others; ++i)
    if (others[i].p && ranges_overlap(out.p, bytes, others[i].p, matrix_bytes(rows, width, others[i].ld, size)))
      return false;
  return true;
}

// Rows as they are, or in 8 bits.
bool rows_ok(const gemm_f32_rows_t* r, long long rows, int width, size_t size) {
  if (!r) return false;
  if (!r->codes) return matrix_ok(r->data, r->ld, width, size) && addressable(rows, r->ld);
  return r->exponents && aligned_to(r->codes, 16) && aligned_to(r->exponents, 16) && r->ld_codes % 16 == 0 &&
         r->ld_exponents % 16 == 0 && r->ld_codes >= (width + 31LL) / 32 * 32 && r->ld_exponents >= (width + 31LL) / 32 &&
         addressable(rows, r->ld_codes) && addressable(rows, r->ld_exponents);
}

bool apart_from_saved(const Matrix& out, const gemm_f32_rows_t* r, long long rows, int width, size_t size) {
  if (!out.p || !r || !r->codes) return true;
  const size_t bytes = matrix_bytes(rows, width, out.ld, size);
  return !ranges_overlap(out.p, bytes, r->codes, static_cast<size_t>(rows) * r->ld_codes) &&
         !ranges_overlap(out.p, bytes, r->exponents, static_cast<size_t>(rows) * r->ld_exponents);
}

RowPlan plan_of(const gemm_f32_block_t& b) {
  RowPlan plan = {};
  plan.width = b.width;
  plan.rows = b.rows;
  return plan;
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" int gemm_f32_block_norm(const gemm_f32_block_t* block, const void* branch, long long ld_branch,
                                   const void* residual, long long ld_residual, void* y, long long ldy, void* h,
                                   long long ldh, float* stats, gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!block_ok(block) || !std::isfinite(block->eps) || block->eps < 0.0f) return GEMM_F32_EINVAL;
  if (block->rows == 0) return GEMM_F32_OK;
  const gemm_f32_block_t& b = *block;
  const size_t es = type_size(b.type);
  const Matrix in[3] = {{branch, ld_branch}, {residual, ld_residual}, {b.ld_gate ? b.gate : nullptr, b.ld_gate}};
  const Matrix out[2] = {{y, ldy}, {h, ldh}};
  for (int i = 0; i < 2; ++i)
    if (!matrix_ok(in[i].p, in[i].ld, b.width, es) || !addressable(b.rows, in[i].ld)) return GEMM_F32_EINVAL;
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && !h) continue;
    if (!matrix_ok(out[i].p, out[i].ld, b.width, es) || !addressable(b.rows, out[i].ld)) return GEMM_F32_EINVAL;
    if (!output_fits(out[i], in, 3, out + 1, i == 0 ? 1 : 0, b.rows, b.width, es)) return GEMM_F32_EINVAL;
  }
  if (!aligned_to(stats, 4)) return GEMM_F32_EINVAL;
  BlockArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.plan = plan_of(b);
  bool aligned = true;
  for (int i = 0; i < 3; ++i) {
    a.in[i] = source(in[i].p, in[i].ld, static_cast<int>(es), a.plan);
    aligned = aligned && (!in[i].p || vector_rows(in[i].p, in[i].ld, b.width, es));
  }
  for (int i = 0; i < 2; ++i) aligned = aligned && (!out[i].p || vector_rows(out[i].p, out[i].ld, b.width, es));
  const int vectors = vectors_of(b, true, a.vectors);
  a.rms = b.norm == GEMM_F32_NORM_RMS;
  a.post = b.post;
  a.gate = gate_of(b);
  a.eps = b.eps;
  a.alpha = b.residual_scale;
  a.beta = b.branch_scale;
  a.y = {y, ldy};
  a.h = {h, ldh};
  a.stats = stats;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  const char* kernel = "none";
  const int rc = b.type == GEMM_F32_TYPE_F32 ? forward<float>(a, vectors, aligned, device, num_sms, stream, &kernel)
                                             : forward<bf16>(a, vectors, aligned, device, num_sms, stream, &kernel);
  if (rc == GEMM_F32_OK) note_launches(1, kernel);
  return rc;
}

extern "C" int gemm_f32_block_norm_grad(const gemm_f32_block_t* block, const void* dy, long long lddy, const void* dh,
                                        long long lddh, const gemm_f32_rows_t* h, const gemm_f32_rows_t* branch,
                                        const float* stats, void* dbranch, long long ld_dbranch, void* dresidual,
                                        long long ld_dresidual, void* dgate, long long ld_dgate, void* dweight,
                                        void* dbias, void* dpost_weight, void* dpost_bias,
                                        gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!block_ok(block)) return GEMM_F32_EINVAL;
  const gemm_f32_block_t& b = *block;
  const size_t es = type_size(b.type), ws = type_size(b.weight_type);
  const int gate = gate_of(b);
  const bool needs_branch = b.post || gate != kNoGate;
  if (b.norm == GEMM_F32_NORM_RMS && (dbias || dpost_bias)) return GEMM_F32_EINVAL;
  if ((!b.post && (dpost_weight || dpost_bias)) || (gate == kNoGate && dgate)) return GEMM_F32_EINVAL;
  void* const vectors_out[kSums] = {dweight, dbias, gate == kChannelGate ? dgate : nullptr, dpost_weight, dpost_bias};
  for (void* v : vectors_out)
    if (!aligned_to(v, ws)) return GEMM_F32_EINVAL;
  const Matrix out[3] = {{dbranch, ld_dbranch}, {dresidual, ld_dresidual}, {gate == kElementGate ? dgate : nullptr, ld_dgate}};
  if (b.rows > 0) {
    if (!matrix_ok(dy, lddy, b.width, es) || !addressable(b.rows, lddy)) return GEMM_F32_EINVAL;
    if (dh && (!matrix_ok(dh, lddh, b.width, es) || !addressable(b.rows, lddh))) return GEMM_F32_EINVAL;
    if (!rows_ok(h, b.rows, b.width, es) || (needs_branch && !rows_ok(branch, b.rows, b.width, es))) return GEMM_F32_EINVAL;
    if (!stats || !aligned_to(stats, 4)) return GEMM_F32_EINVAL;
    const gemm_f32_rows_t* const used = needs_branch ? branch : nullptr;
    const Matrix in[5] = {{dy, lddy}, {dh, lddh}, {h->codes ? nullptr : h->data, h->ld},
                          {used && !used->codes ? used->data : nullptr, used ? used->ld : 0},
                          {gate == kElementGate ? b.gate : nullptr, b.ld_gate}};
    for (int i = 0; i < 3; ++i) {
      if (!out[i].p) continue;
      if (!matrix_ok(out[i].p, out[i].ld, b.width, es) || !addressable(b.rows, out[i].ld)) return GEMM_F32_EINVAL;
      if (!output_fits(out[i], in, 5, out + i + 1, 2 - i, b.rows, b.width, es)) return GEMM_F32_EINVAL;
      if (!apart_from_saved(out[i], h, b.rows, b.width, es) || !apart_from_saved(out[i], used, b.rows, b.width, es))
        return GEMM_F32_EINVAL;
    }
  }
  bool wanted = false;
  for (void* v : vectors_out) wanted = wanted || v;
  if (!wanted && (b.rows == 0 || !(out[0].p || out[1].p || out[2].p))) return GEMM_F32_OK;
  BlockGradArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.plan = plan_of(b);
  bool aligned = true;
  if (b.rows > 0) {
    const int size = static_cast<int>(es);
    auto add = [&](int i, const void* p, long long ld) {
      a.in[i] = source(p, ld, size, a.plan);
      aligned = aligned && (!p || vector_rows(p, ld, b.width, es));
    };
    auto add_rows = [&](int i, int exponents, const gemm_f32_rows_t* r) {
      if (!r->codes) return add(i, r->data, r->ld);
      a.in[i] = saved_source(r->codes, r->ld_codes, false, a.plan);
      a.in[exponents] = saved_source(r->exponents, r->ld_exponents, true, a.plan);
    };
    add(kGradDy, dy, lddy);
    add(kGradDh, dh, lddh);
    add_rows(kGradH, kGradHExponents, h);
    if (needs_branch) add_rows(kGradBranch, kGradBranchExponents, branch);
    if (gate == kElementGate) add(kGradGate, b.gate, b.ld_gate);
    for (const Matrix& o : out) aligned = aligned && (!o.p || vector_rows(o.p, o.ld, b.width, es));
    // codes alone are always on boundaries, but the vectors are those of whole rows
    aligned = aligned && b.width * es % 16 == 0;
  }
  const int vectors = vectors_of(b, false, a.vectors);
  a.rms = b.norm == GEMM_F32_NORM_RMS;
  a.post = b.post;
  a.gate = gate;
  a.branch = needs_branch;
  a.alpha = b.residual_scale;
  a.beta = b.branch_scale;
  a.stats = stats;
  a.dbranch = {const_cast<void*>(out[0].p), out[0].ld};
  a.dresidual = {const_cast<void*>(out[1].p), out[1].ld};
  a.dgate = {const_cast<void*>(out[2].p), out[2].ld};
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  int launches = 0;
  const char* kernel = "none";
  const WorkspaceCall call;
  const int rc = b.type == GEMM_F32_TYPE_F32
                     ? gradient<float>(a, vectors_out, vectors, aligned, b.weight_type, device, num_sms, stream, &launches, &kernel)
                     : gradient<bf16>(a, vectors_out, vectors, aligned, b.weight_type, device, num_sms, stream, &launches, &kernel);
  if (rc == GEMM_F32_OK) note_launches(launches, kernel);
  return rc;
}
