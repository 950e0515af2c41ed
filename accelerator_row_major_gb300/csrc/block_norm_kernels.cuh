// The norms at a block's ends, with its gate and residual, and their
// gradients: the kernels (sm_103a).  Included once per element type.
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
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/gemm_f32_block.h"
#include "block_norm.h"
#include "block_plan.h"
#include "block_rows.cuh"
#include "device_common.cuh"
#include "launch.h"
#include "row_common.cuh"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

__device__ __forceinline__ Pair both(float x) { return pair_of(x, x); }

template <class T>
__device__ __forceinline__ bool output_ok(const Output& o, const RowPlan& plan, long long row, unsigned* err) {
  return GEMM_IN_EXTENT(row * o.ld + plan.width - 1, stored_extent(plan.rows, plan.width, o.ld), err,
                        kSiteBoundsRows);
}

// The vectors into shared memory, by the threads that compute: of four columns
// all vectors' values are on their way before the first is stored (value by
// value, vector after vector, this took 5 us for each vector of 4096).
template <class T, class Part>
__device__ __forceinline__ void fill_vectors(float* columns, const VectorArgs& a, const RowPlan& plan,
                                             const RingPlace& ring) {
  const int threads = plan.groups * plan.lanes, slots = Part::slots(plan.lanes);
  if (static_cast<int>(threadIdx.x) >= threads) return;
  for (int slot = 4 * threadIdx.x; slot < slots; slot += 4 * threads) {
    float f[kVectors][4];
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      if (a.slot[v] < 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = Part::column_of_slot(slot + j);
        f[v][j] = c >= ring.width ? 0.0f
                  : a.p[v]        ? vector_value<T>(a.p[v], a.f32, ring.col0 + c)
                                  : (v == kWeight || v == kPostWeight ? 1.0f : 0.0f);
        if (v == kPostWeight && a.joined && a.p[kGateVector] && c < ring.width)
          f[v][j] *= vector_value<T>(a.p[kGateVector], a.f32, ring.col0 + c);
      }
    }
#pragma unroll
    for (int v = 0; v < kVectors; ++v)
      if (a.slot[v] >= 0)
        *reinterpret_cast<float4*>(columns + a.slot[v] * slots + slot) = make_float4(f[v][0], f[v][1], f[v][2], f[v][3]);
  }
}

// 16 warps compute with 112 registers a thread, some of them left by the
// warpgroup of the producers: in a plain launch of as many there would be 96.
constexpr int kProducerRegisters = 32, kComputeRegisters = 112;
static_assert(kProducerThreads * kProducerRegisters + 32 * kRowWarps * kComputeRegisters <=
                  96 * (kProducerThreads + 32 * kRowWarps),
              "registers of a launch of 96 a thread");
constexpr int kComputeBarrier = 15;      // of the threads that compute; no group has it (at most 8 groups meet at theirs)

// The producer's warpgroup, to its end.
template <bool ALIGNED, int N>
__device__ __forceinline__ void producer_warps(const RowSource (&in)[N], const RowPlan& plan, const RingPlace& ring,
                                               const float* stats, uint32_t stats_mask, unsigned* err) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegisters));
  const int warp = static_cast<int>(threadIdx.x - (blockDim.x - kProducerThreads)) / 32;
  produce_rows<ALIGNED>(in, plan, ring, stats, stats_mask, err, warp, [] { __syncthreads(); });
  if (plan.ctas > 1) cluster_sync();
}

// ---------------------------------------------------------------- forward
template <class T, int NE, bool VEC>
__global__ void __launch_bounds__(kProducerThreads + 32 * kRowWarps, 1)
    block_norm_kernel(const __grid_constant__ BlockArgs a) {
  using Part = RowPart<T, NE, VEC>;
  constexpr int NP = Part::NP, NC = Part::NC, CP = Part::CP;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ RowShared shared;
  const RowPlan& plan = a.plan;
  const int rank = plan.ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const RingPlace ring(plan, smem_rows, rank);
  if (threadIdx.x == 0) {
    if (plan.ctas > 1) RowSums::init(shared, plan);
    ring.init(plan);
  }
  __syncthreads();
  if (plan.ctas > 1) cluster_sync();     // every CTA of the cluster runs
  grid_launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x >= blockDim.x - kProducerThreads) {
    producer_warps<VEC>(a.in, plan, ring, nullptr, 0u, a.err);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegisters));
  const int group = threadIdx.x / plan.lanes, t = threadIdx.x % plan.lanes;
  float* const columns = reinterpret_cast<float*>(smem_rows);
  fill_vectors<T, Part>(columns, a.vectors, plan, ring);
  __syncthreads();
  const Part mine(t, ring.width);
  const bool full = mine.full();
  const float inv = 1.0f / static_cast<float>(plan.width);
  const auto vector = [&](int v) { return columns + a.vectors.slot[v] * Part::slots(plan.lanes); };
  RowSums sums = {shared, plan, a.err, group, t, rank};
  // x around its mean (0 for rms), 1 / its root mean square there.
  const auto normalise = [&](Pair(&x)[NP], float& mean, float& rstd) {
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
      if (!full) {
#pragma unroll
        for (int v = 0; v < NC; ++v) mine.drop(v, x + v * CP);
      }
    }
    Pair sum = 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) sum = fma2(x[j], x[j], sum);
    s[0] = sum_of(sum);
    sums.add<1>(s);
    rstd = rsqrtf(s[0] * inv + a.eps);
  };
  // f(j, value) for every pair of elements, of a vector or of a row
  const auto each = [&](int vector_at, auto f) {
    const float* const from = vector(vector_at);
#pragma unroll
    for (int v = 0; v < NC; ++v) {
      Pair w[CP];
      mine.columns(from, v, w);
#pragma unroll
      for (int k = 0; k < CP; ++k) f(v * CP + k, w[k]);
    }
  };
  const auto each_of = [&](const uint8_t* row, auto f) {
#pragma unroll
    for (int v = 0; v < NC; ++v) {
      Pair w[CP];
      mine.load(row, v, w);
#pragma unroll
      for (int k = 0; k < CP; ++k) f(v * CP + k, w[k]);
    }
  };
  const auto store = [&](const Output& o, long long row, const Pair(&x)[NP]) {
    if (!o.p || !output_ok<T>(o, plan, row, a.err)) return;
    T* const to = static_cast<T*>(o.p) + row * o.ld + ring.col0;
#pragma unroll
    for (int v = 0; v < NC; ++v) {
      Pair w[CP];
#pragma unroll
      for (int k = 0; k < CP; ++k) w[k] = x[v * CP + k];
      mine.store(to, v, w);
    }
  };

  RingReader reader(ring, plan, a.err, group);
  long long row = group < plan.groups ? ring.first * plan.turn + group : plan.rows;
  for (; row < plan.rows; row += ring.step * plan.turn) {
    reader.wait();
    Pair x[NP];
    float mean, rstd, mean_b = 0.0f, rstd_b = 0.0f;
    each_of(reader.at(a.in[kInBranch], row, 0, VEC), [&](int j, Pair v) { x[j] = v; });
    if (a.post) {
      normalise(x, mean_b, rstd_b);
      each(kPostWeight, [&](int j, Pair w) { x[j] = mul2(mul2(x[j], both(rstd_b)), w); });
      if (a.vectors.slot[kPostBias] >= 0) each(kPostBias, [&](int j, Pair w) { x[j] = add2(x[j], w); });
    }
    if (a.gate == kElementGate)
      each_of(reader.at(a.in[kInGate], row, 0, VEC), [&](int j, Pair w) { x[j] = mul2(x[j], w); });
    else if (a.gate == kChannelGate)
      each(kGateVector, [&](int j, Pair w) { x[j] = mul2(x[j], w); });
    each_of(reader.at(a.in[kInResidual], row, 0, VEC),
            [&](int j, Pair w) { x[j] = fma2(x[j], both(a.beta), mul2(w, both(a.alpha))); });
    reader.release();
    store(a.h, row, x);                  // an h that is an input: all of this row has been read
    normalise(x, mean, rstd);
    each(kWeight, [&](int j, Pair w) { x[j] = mul2(mul2(x[j], both(rstd)), w); });
    if (a.vectors.slot[kBias] >= 0) each(kBias, [&](int j, Pair w) { x[j] = add2(x[j], w); });
    store(a.y, row, x);
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
// LAYER: around the means; POST: the branch was normed; CHANNEL: a gate per
// channel (a gate per element is the launch's choice).  What a form does not
// have costs no registers.  With POST and CHANNEL the sums over the rows are
// of d and d hat_b: the gate, the same for all rows, and the weights come to
// them at the end (dpost_weight = gate sum d hat_b, dpost_bias = gate sum d,
// dgate = post_weight sum d hat_b + post_bias sum d): two sums for three and
// one vector, gate post_weight, for three on the way, which leaves room for two
// rows at a time (layer norms, 8192 columns: 4096 rows of bfloat16 126 us, 151
// with one row at a time; 8192 of fp32 334 -> 280 with the fewer sums, 282 now).
template <class T, int NE, int ROWS, bool VEC, bool LAYER, bool POST, bool CHANNEL>
__global__ void __launch_bounds__(kProducerThreads + 32 * kRowWarps, 1)
    block_norm_grad_kernel(const __grid_constant__ BlockGradArgs a) {
  using Part = RowPart<T, NE, VEC>;
  constexpr int NP = Part::NP, NC = Part::NC, CP = Part::CP;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ RowShared shared;
  const RowPlan& plan = a.plan;
  const int rank = plan.ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const RingPlace ring(plan, smem_rows, rank);
  if (threadIdx.x == 0) {
    if (plan.ctas > 1) RowSums::init(shared, plan);
    ring.init(plan);
  }
  __syncthreads();
  if (plan.ctas > 1) cluster_sync();     // every CTA of the cluster runs
  grid_launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x >= blockDim.x - kProducerThreads) {
    producer_warps<VEC>(a.in, plan, ring, a.stats, (LAYER ? 3u : 2u) * (POST ? 5u : 1u), a.err);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegisters));
  const int group = threadIdx.x / plan.lanes, t = threadIdx.x % plan.lanes;
  float* const columns = reinterpret_cast<float*>(smem_rows);
  fill_vectors<T, Part>(columns, a.vectors, plan, ring);
  __syncthreads();
  const Part mine(t, ring.width);
  const bool full = mine.full();
  const float inv = 1.0f / static_cast<float>(plan.width);
  const auto vector = [&](int v) { return columns + a.vectors.slot[v] * Part::slots(plan.lanes); };
  RowSums sums = {shared, plan, a.err, group, t, rank};
  constexpr bool kJoined = POST && CHANNEL;
  Pair total[kSums][NP];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int j = 0; j < NP; ++j) total[k][j] = 0;
  // The two means over a row of a norm's gradient, of the gradients `ones` and
  // of their products with hat, negative.
  const auto means = [&](const Pair(&ones)[ROWS], const Pair(&along)[ROWS], float(&c1)[ROWS], float(&c2)[ROWS]) {
    constexpr int N = LAYER ? 2 : 1;
    float v[N * ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      v[N * r] = sum_of(along[r]);
      if (LAYER) v[N * r + N - 1] = sum_of(ones[r]);
    }
    sums.add<N * ROWS>(v);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      c1[r] = LAYER ? -v[N * r + N - 1] * inv : 0.0f;
      c2[r] = -v[N * r] * inv;
    }
  };
  const auto store = [&](const Output& o, long long row, const Pair(&x)[NP], float by) {
    if (!o.p || row >= plan.rows || !output_ok<T>(o, plan, row, a.err)) return;
    T* const to = static_cast<T*>(o.p) + row * o.ld + ring.col0;
    const auto all = [&](auto scaled) {
#pragma unroll
      for (int v = 0; v < NC; ++v) {
        Pair w[CP];
#pragma unroll
        for (int k = 0; k < CP; ++k) w[k] = decltype(scaled)::value ? mul2(x[v * CP + k], both(by)) : x[v * CP + k];
        mine.store(to, v, w);
      }
    };
    if (by == 1.0f)
      all(std::false_type{});
    else
      all(std::true_type{});
  };
  // f(r, v, loader) for every row r and chunk v, the loader filling a chunk of
  // the row of h or of the branch, which is as it is or in 8 bits.  What a turn
  // has no row for counts as zeros.
  const auto rows_of = [&](const RingReader& reader, long long row, int at, int exponents_at, auto f) {
    const uint8_t* from[ROWS];
    const uint8_t* exponents[ROWS];
    const bool saved = a.in[exponents_at].p != nullptr;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      from[r] = reader.at(a.in[at], row + r, r, VEC || saved);
      exponents[r] = saved ? reader.at(a.in[exponents_at], row + r, r, true) : nullptr;
    }
    if (saved)
      f([&](int r, int v, Pair(&x)[CP]) { mine.load_saved(from[r], exponents[r], v, x); });
    else
      f([&](int r, int v, Pair(&x)[CP]) { mine.load(from[r], v, x); });
  };

  // Both norms take sums over the row, one after the other.  With a gate per
  // element, the second ones go with the next row's first: one exchange a row,
  // of the same sums, what the end of a row needs in registers meanwhile
  // (4096 x 8192 bfloat16 163 -> 143 us).  Where two rows fit instead, they are
  // as good, and a wide fp32 row has no room for both (8192 x 8192, a gate per
  // channel, 302 with it, 280 without).
  constexpr bool kLate = LAYER && POST && !CHANNEL;
  constexpr int kLatePairs = kLate ? NP : 1;
  Pair late_e[kLatePairs], late_hat[kLatePairs], late_se = 0, late_seh = 0;
  float late_rstd = 0.0f;
  long long late_row = -1;               // none
  // dbranch of the row r: e through the branch's norm
  const auto end_row = [&](Pair* e, const Pair* hat_b, float rstd_b, float c1, float c2) {
    const float by = rstd_b * a.beta;
#pragma unroll
    for (int j = 0; j < NP; ++j)
      e[j] = fma2(e[j], both(by), LAYER ? fma2(hat_b[j], both(c2 * by), both(c1 * by)) : mul2(hat_b[j], both(c2 * by)));
  };

  // A norm's hat, of pair k of chunk v, from what is left of x without the mean:
  // x rstd - mean rstd would be off by a rounding of mean rstd, however small hat
  // is, and leave the range where hat does not.  0 outside the row.
  const auto normed = [&](int v, int k, Pair x, float mean, float rstd) {
    return mul2(LAYER ? add2(x, mine.within(v, k, -mean)) : x, both(rstd));
  };
  const auto nothing = [](Pair(&x)[CP]) {
#pragma unroll
    for (int k = 0; k < CP; ++k) x[k] = 0;
  };

  RingReader reader(ring, plan, a.err, group * ROWS);
  long long row = group < plan.groups ? ring.first * plan.turn + group * ROWS : plan.rows;
  for (; row < plan.rows; row += ring.step * plan.turn) {
    reader.wait();
    const bool whole = ROWS == 1 || row + ROWS <= plan.rows;
    const auto there = [&](int r) { return r == 0 || whole; };
    float mean[ROWS], rstd[ROWS], mean_b[ROWS], rstd_b[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float4 stats = reader.stats(r);
      mean[r] = there(r) ? stats.x : 0.0f;
      rstd[r] = there(r) ? stats.y : 0.0f;
      mean_b[r] = there(r) ? stats.z : 0.0f;
      rstd_b[r] = there(r) ? stats.w : 0.0f;
    }
    Pair hat[ROWS][NP], g[ROWS][NP], sg[ROWS], sgh[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sg[r] = sgh[r] = 0;
    rows_of(reader, row, kGradH, kGradHExponents, [&](auto load_h) {
      const uint8_t* dy[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) dy[r] = reader.at(a.in[kGradDy], row + r, r, VEC);
      const float* const weight = vector(kWeight);
#pragma unroll
      for (int v = 0; v < NC; ++v) {
        Pair w[CP];
        mine.columns(weight, v, w);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          Pair x[CP], y[CP];
          if (there(r)) {
            load_h(r, v, x);
            mine.load(dy[r], v, y);
          } else {
            nothing(x);
            nothing(y);
          }
#pragma unroll
          for (int k = 0; k < CP; ++k) {
            const int j = v * CP + k;
            hat[r][j] = normed(v, k, x[k], mean[r], rstd[r]);
            total[kSumWeight][j] = fma2(y[k], hat[r][j], total[kSumWeight][j]);
            if (LAYER) total[kSumBias][j] = add2(total[kSumBias][j], y[k]);
            g[r][j] = mul2(y[k], w[k]);
            if (LAYER) sg[r] = add2(sg[r], g[r][j]);
            sgh[r] = fma2(g[r][j], hat[r][j], sgh[r]);
          }
        }
      }
    });
    float c1[ROWS], c2[ROWS];
    if constexpr (kLate) {
      float v[4] = {sum_of(sgh[0]), sum_of(sg[0]), sum_of(late_seh), sum_of(late_se)};
      sums.add<4>(v);
      c1[0] = -v[1] * inv;
      c2[0] = -v[0] * inv;
      if (late_row >= 0) {
        end_row(late_e, late_hat, late_rstd, -v[3] * inv, -v[2] * inv);
        store(a.dbranch, late_row, late_e, 1.0f);
      }
    } else {
      means(sg, sgh, c1, c2);
    }
    // d = dh + rstd (g + c1 + hat c2), in place of g
    Pair(&d)[ROWS][NP] = g;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
      for (int j = 0; j < NP; ++j)
        d[r][j] = fma2(g[r][j], both(rstd[r]),
                       LAYER ? fma2(hat[r][j], both(c2[r] * rstd[r]), both(c1[r] * rstd[r])) : mul2(hat[r][j], both(c2[r] * rstd[r])));
      if (a.in[kGradDh].p && there(r)) {
        const uint8_t* const dh = reader.at(a.in[kGradDh], row + r, r, VEC);
#pragma unroll
        for (int v = 0; v < NC; ++v) {
          Pair x[CP];
          mine.load(dh, v, x);
#pragma unroll
          for (int k = 0; k < CP; ++k) d[r][v * CP + k] = add2(d[r][v * CP + k], x[k]);
        }
      }
      // an output that is an input: the ring has all of this row
      store(a.dresidual, row + r, d[r], a.alpha);
    }
    if (!(POST || CHANNEL) && a.gate == kNoGate) {
      reader.release();
#pragma unroll
      for (int r = 0; r < ROWS; ++r) store(a.dbranch, row + r, d[r], a.beta);
      continue;
    }
    if (!full) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int v = 0; v < NC; ++v) mine.drop(v, d[r] + v * CP);
    }
    // e = d gate (joined to the post weight where that is a vector), without
    // beta: what is linear in it gets that at its end
    Pair(&hat_b)[ROWS][NP] = hat;        // the branch's in place of h's
    Pair se[ROWS], seh[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) se[r] = seh[r] = 0;
    const auto through_gate = [&](auto load_branch, auto element) {
      constexpr bool kElement = decltype(element)::value, kGated = (CHANNEL && !kJoined) || kElement;
      const bool bias = POST && LAYER && kGated && a.vectors.slot[kPostBias] >= 0;
      const uint8_t* gate[ROWS];
      T* to[ROWS];
      const bool stores = kElement && a.dgate.p;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        gate[r] = kElement ? reader.at(a.in[kGradGate], row + r, r, VEC) : nullptr;
        to[r] = static_cast<T*>(a.dgate.p) + (row + r) * a.dgate.ld + ring.col0;
      }
#pragma unroll
      for (int v = 0; v < NC; ++v) {
        Pair w[CP], post_bias[CP], channel[CP];
        if (POST) mine.columns(vector(kPostWeight), v, w);
        if (kGated && POST) {
          if (bias) {
            mine.columns(vector(kPostBias), v, post_bias);
          } else {
            nothing(post_bias);
          }
        }
        if (CHANNEL && !kJoined) mine.columns(vector(kGateVector), v, channel);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          Pair x[CP];
          Pair* const e = d[r] + v * CP;
          if (there(r))
            load_branch(r, v, x);
          else
            nothing(x);
          if (POST) {
#pragma unroll
            for (int k = 0; k < CP; ++k) x[k] = hat_b[r][v * CP + k] = normed(v, k, x[k], mean_b[r], rstd_b[r]);
          }
          if (kGated) {
            Pair p[CP], by[CP];
#pragma unroll
            for (int k = 0; k < CP; ++k) p[k] = POST ? fma2(x[k], w[k], post_bias[k]) : x[k];
            if (CHANNEL) {
#pragma unroll
              for (int k = 0; k < CP; ++k) by[k] = channel[k];
            } else if (there(r)) {
              mine.load(gate[r], v, by);
            } else {
              nothing(by);
            }
#pragma unroll
            for (int k = 0; k < CP; ++k) {
              if (CHANNEL)
                total[kSumGate][v * CP + k] = fma2(e[k], p[k], total[kSumGate][v * CP + k]);
              else
                p[k] = mul2(mul2(e[k], p[k]), both(a.beta));
              e[k] = mul2(e[k], by[k]);
            }
            if (stores && there(r) && output_ok<T>(a.dgate, plan, row + r, a.err)) mine.store(to[r], v, p);
          }
          if (POST) {
#pragma unroll
            for (int k = 0; k < CP; ++k) {
              const int j = v * CP + k;
              total[kSumPostWeight][j] = fma2(e[k], x[k], total[kSumPostWeight][j]);
              if (LAYER) total[kSumPostBias][j] = add2(total[kSumPostBias][j], e[k]);
              e[k] = mul2(e[k], w[k]);
              if (LAYER) se[r] = add2(se[r], e[k]);
              seh[r] = fma2(e[k], x[k], seh[r]);
            }
          }
        }
      }
    };
    rows_of(reader, row, kGradBranch, kGradBranchExponents, [&](auto load_branch) {
      if (!CHANNEL && a.gate == kElementGate)
        through_gate(load_branch, std::integral_constant<bool, !CHANNEL>{});
      else
        through_gate(load_branch, std::false_type{});
    });
    reader.release();
    if constexpr (kLate) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        late_e[j] = d[0][j];
        late_hat[j] = hat_b[0][j];
      }
      late_se = se[0];
      late_seh = seh[0];
      late_rstd = rstd_b[0];
      late_row = row;
    } else {
      if (POST) means(se, seh, c1, c2);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (POST) end_row(d[r], hat_b[r], rstd_b[r], c1[r], c2[r]);
        store(a.dbranch, row + r, d[r], POST ? 1.0f : a.beta);
      }
    }
  }
  if constexpr (kLate) {
    if (late_row >= 0) {                 // the group's, on every CTA of the cluster
      Pair se[1] = {late_se}, seh[1] = {late_seh};
      float c1[1], c2[1];
      means(se, seh, c1, c2);
      end_row(late_e, late_hat, late_rstd, c1[0], c2[0]);
      store(a.dbranch, late_row, late_e, 1.0f);
    }
  }
  if (plan.ctas > 1) cluster_sync();     // no CTA leaves while another may write to it
  if (!a.sums) return;
  // The groups' sums, added in group order: one row of partials per CTA (or
  // cluster) and vector; what was the ring makes room for those of all groups.
  const int threads = static_cast<int>(blockDim.x) - kProducerThreads, slots = Part::slots(plan.lanes);
  const auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"n"(kComputeBarrier), "r"(threads) : "memory"); };
  meet();
  if (group < plan.groups) {
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      const bool there = k == kSumWeight || (k == kSumBias && LAYER) || (k == kSumGate && CHANNEL) ||
                         (k == kSumPostWeight && POST) || (k == kSumPostBias && POST && LAYER);
      if (!there || a.sum[k] < 0) continue;
#pragma unroll
      for (int q = 0; q < NE / 4; ++q) {
        const Pair by = both(k == kSumWeight || k == kSumBias ? 1.0f : a.beta);
        if (kJoined && (k == kSumGate || k == kSumPostWeight || k == kSumPostBias)) {
          // sums of d and d hat_b become those of the vectors
          const int base = mine.slot(q);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const auto pair = [&](int vector, float otherwise) {
              float f[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int c = Part::column_of_slot(base + 2 * j + i);
                f[i] = c < ring.width && a.vectors.p[vector] ? vector_value<T>(a.vectors.p[vector], a.vectors.f32, ring.col0 + c)
                                                             : otherwise;
              }
              return pair_of(f[0], f[1]);
            };
            if (k == kSumGate) {
              const Pair along = mul2(pair(kPostWeight, 1.0f), total[kSumPostWeight][2 * q + j]);
              total[kSumGate][2 * q + j] =
                  LAYER ? fma2(pair(kPostBias, 0.0f), total[kSumPostBias][2 * q + j], along) : along;
            } else {
              total[k][2 * q + j] = mul2(pair(kGateVector, 1.0f), total[k][2 * q + j]);
            }
          }
        }
        float4 f;
        unpair(mul2(total[k][2 * q], by), f.x, f.y);
        unpair(mul2(total[k][2 * q + 1], by), f.z, f.w);
        *reinterpret_cast<float4*>(columns + (a.sum[k] * plan.groups + group) * slots + mine.slot(q)) = f;
      }
    }
  }
  meet();
  float* const to = a.partials + static_cast<size_t>(blockIdx.x / plan.ctas) * a.sums * a.ld_partials + ring.col0;
  for (int k = 0; k < a.sums; ++k) {
    for (int slot = 4 * threadIdx.x; slot < slots; slot += 4 * threads) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int i = 0; i < plan.groups; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(columns + (k * plan.groups + i) * slots + slot);
        v.x += f.x;
        v.y += f.y;
        v.z += f.z;
        v.w += f.w;
      }
      const float values[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = Part::column_of_slot(slot + j);
        if (col < ring.width) to[k * a.ld_partials + col] = values[j];
      }
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
  return vector_value<T>(a.p[v], a.f32, d);
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
        float* const to = a.partials + (static_cast<size_t>(blockIdx.x) * a.sums + a.sum[k]) * a.ld_partials + d;
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
// Partial sums of 128 columns of one vector: chains of every 16th CTA, then the
// chains in order.
struct ColumnArgs {
  const float* partials;
  long long ld;
  void* out[kSums];                      // by their place in the partials
  int sums, ctas, width;
};

constexpr int kColumnChains = 16;

template <class WT>
__global__ void __launch_bounds__(32 * kColumnChains) block_columns_kernel(const __grid_constant__ ColumnArgs a) {
  __shared__ float4 chains[kColumnChains][32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, chain = threadIdx.x >> 5, k = blockIdx.y;
  const long long d = blockIdx.x * 128LL + 4 * lane;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (d < a.width) {                     // a row of partials has whole vectors
    const float* from = a.partials + (static_cast<size_t>(chain) * a.sums + k) * a.ld + d;
#pragma unroll 10
    for (int c = chain; c < a.ctas; c += kColumnChains, from += kColumnChains * a.sums * a.ld) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(from));
      v.x += f.x;
      v.y += f.y;
      v.z += f.z;
      v.w += f.w;
    }
  }
  chains[chain][lane] = v;
  __syncthreads();
  if (threadIdx.x < 128 && blockIdx.x * 128LL + threadIdx.x < a.width) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kColumnChains; ++c) s += reinterpret_cast<const float*>(chains[c])[threadIdx.x];
    static_cast<WT*>(a.out[k])[blockIdx.x * 128LL + threadIdx.x] = from_f32<WT>(s);
  }
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

// Sets a kernel's shared memory up, once per device, and launches it; where
// CTAs form clusters, with no more of them than run at once (`grid` is
// reduced to that).
template <auto Kernel, class Args>
int launch_rows(const Args& a, int threads, int device, int* grid, size_t bytes, cudaStream_t stream) {
  static std::atomic<int> clusters[kMaxDevices][4];   // at a time, per log2 of their CTAs; 1 for single CTAs
  const RowPlan& plan = a.plan;
  std::atomic<int>& kept = clusters[device % kMaxDevices][plan.ctas == 1 ? 0 : plan.ctas == 2 ? 1 : plan.ctas == 4 ? 2 : 3];
  int most = kept.load();
  cudaLaunchConfig_t config = {};
  config.blockDim = dim3(threads);
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
      full.dynamicSmemBytes = kMostShared;       // one CTA per SM
      full.attrs = attr + 1;
      full.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&most, Kernel, &full) != cudaSuccess || most < 1) {
        (void)cudaGetLastError();
        return GEMM_F32_ELAUNCH;
      }
    }
    kept.store(most);
  }
  if (plan.ctas > 1) *grid = std::min(*grid, most * plan.ctas);
  config.gridDim = dim3(*grid);
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

template <class T, int NE>
int forward_form(const BlockArgs& a, const BlockLaunch& l, Layout<kInputs>& best) {
  const int threads = cta_threads(a.plan);
  return l.aligned ? launch_rows<block_norm_kernel<T, NE, true>>(a, threads, l.device, &best.grid, best.bytes, l.stream)
                   : launch_rows<block_norm_kernel<T, NE, false>>(a, threads, l.device, &best.grid, best.bytes, l.stream);
}

template <class T>
int forward(BlockArgs& a, const BlockLaunch& l) {
  const Lane lanes[3] = {{8, 1}, {16, 1}, {32, 1}};
  Layout<kInputs> best = best_layout(a.plan, a.in, lanes, false, 0, l);
  ++*l.launches;
  if (best.lane.ne == 0) {
    *l.kernel = "block_norm_wide_kernel";
    return launch_plain(block_norm_wide_kernel<T>, dim3(static_cast<unsigned>(std::min<long long>(a.plan.rows, 4LL * l.num_sms))),
                        kWideThreads, l.stream, a);
  }
  *l.kernel = "block_norm_kernel";
  a.plan = best.plan;
  std::copy(best.in, best.in + kInputs, a.in);
  if (best.lane.ne == 8) return forward_form<T, 8>(a, l, best);
  return best.lane.ne == 16 ? forward_form<T, 16>(a, l, best) : forward_form<T, 32>(a, l, best);
}

template <class T, int NE, int ROWS, bool LAYER, bool POST, bool CHANNEL>
int gradient_form(const BlockGradArgs& a, const BlockLaunch& l, Layout<kGradInputs>& best) {
  const int threads = cta_threads(a.plan);
  return l.aligned ? launch_rows<block_norm_grad_kernel<T, NE, ROWS, true, LAYER, POST, CHANNEL>>(a, threads, l.device, &best.grid,
                                                                                            best.bytes, l.stream)
                   : launch_rows<block_norm_grad_kernel<T, NE, ROWS, false, LAYER, POST, CHANNEL>>(a, threads, l.device, &best.grid,
                                                                                             best.bytes, l.stream);
}

// f with the three choices as template arguments.
template <class F>
int with_form(bool layer, bool post, bool channel, F f) {
  const auto third = [&](auto x, auto y) { return channel ? f(x, y, std::true_type{}) : f(x, y, std::false_type{}); };
  const auto second = [&](auto x) { return post ? third(x, std::true_type{}) : third(x, std::false_type{}); };
  return layer ? second(std::true_type{}) : second(std::false_type{});
}

template <class T>
int gradient(BlockGradArgs& a, void* const (&vectors_out)[kSums], const BlockLaunch& l) {
  ColumnArgs c = {};
  c.width = a.plan.width;
  c.ld = a.ld_partials = (a.plan.width + 3LL) / 4 * 4;
  for (int k = 0; k < kSums; ++k) {
    a.sum[k] = vectors_out[k] ? a.sums++ : -1;
    if (vectors_out[k]) c.out[a.sum[k]] = vectors_out[k];
  }
  int rc = GEMM_F32_OK;
  *l.kernel = "block_columns_kernel";
  if (a.plan.rows > 0) {
    // two layer norms without a gate: the form with a gate of ones, whose sums leave room for two rows (4096 x 8192
    // bfloat16 123 us against 129 with the form of any gate; fp32 rows of 8192 are 10 % faster with that)
    const bool channel = a.gate == kChannelGate || (!a.rms && a.post && a.gate == kNoGate);
    rc = with_form(!a.rms, a.post, channel, [&](auto layer, auto post, auto by_channel) -> int {
      constexpr bool kLayer = decltype(layer)::value, kPost = decltype(post)::value, kChannel = decltype(by_channel)::value;
      constexpr Lane kMore = grad_lane(kLayer, kPost, kChannel);
      const Lane lanes[2] = {{8, 1}, kMore};
      BlockLaunch rows = l;
      if (kPost && kChannel) rows.vectors = 2;             // the weight, and the gate's joined to the post weight
      Layout<kGradInputs> best = best_layout(a.plan, a.in, lanes, true, a.sums, rows);
      c.ctas = best.lane.ne ? best.grid / best.plan.ctas : static_cast<int>(std::min<long long>(a.plan.rows, 2LL * l.num_sms));
      if (a.sums) {
        a.partials = static_cast<float*>(acquire_scratch(
            l.device, l.stream, sizeof(float) * static_cast<size_t>(c.ctas) * a.sums * a.ld_partials));
        if (!a.partials) return GEMM_F32_ESCRATCH;
      }
      ++*l.launches;
      if (best.lane.ne == 0) {
        *l.kernel = "block_norm_grad_wide_kernel";
        return launch_plain(block_norm_grad_wide_kernel<T>, dim3(c.ctas), kWideThreads, l.stream, a);
      }
      *l.kernel = "block_norm_grad_kernel";
      if (kPost && kChannel) {
        const int slots[kVectors] = {0, -1, 1, -1, -1};
        std::copy(slots, slots + kVectors, a.vectors.slot);
        a.vectors.joined = 1;
      }
      a.plan = best.plan;
      std::copy(best.in, best.in + kGradInputs, a.in);
      const bool more = best.lane.ne != 8 || best.lane.rows != 1;
      const int got = more ? gradient_form<T, kMore.ne, kMore.rows, kLayer, kPost, kChannel>(a, l, best)
                           : gradient_form<T, 8, 1, kLayer, kPost, kChannel>(a, l, best);
      c.ctas = best.grid / best.plan.ctas;
      return got;
    });
  }
  if (rc == GEMM_F32_OK && a.sums) {
    c.partials = a.partials;
    c.sums = a.sums;
    const dim3 blocks(static_cast<unsigned>((c.width + 127LL) / 128), a.sums);
    rc = l.weights_f32 ? launch_plain(block_columns_kernel<float>, blocks, 32 * kColumnChains, l.stream, c)
                       : launch_plain(block_columns_kernel<T>, blocks, 32 * kColumnChains, l.stream, c);
    ++*l.launches;
  }
  return rc;
}

}  // namespace
}  // namespace gemm_f32_impl
