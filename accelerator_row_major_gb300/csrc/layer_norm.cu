// Layer norm over the rows of a matrix and its gradient (sm_103a).
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//   hat  = (x - mean) rstd,  y = hat weight + bias
//   g    = dy weight,  dx = rstd (g - sum(g)/D - hat sum(g hat)/D)
//   dweight = sum over rows of dy hat,  dbias = sum over rows of dy
//
// Both passes are bound by memory traffic: x in and y out, or dy and x in
// and dx out, each once.  So a row is held in the registers of the threads
// that share it from its load to its result: the mean, then the sum of the
// centred squares, then y (or the two sums of the gradient, then dx) come
// from the same registers.  The gradient's grid is persistent: a thread
// keeps the same columns for all of its rows and sums their dy hat and dy in
// registers, so the column sums cost no traffic but one row of partials per
// CTA, which a second kernel adds in CTA order (no atomics: the result does
// not depend on timing).
//
// Many rows are streamed (layer_norm_stream.cuh): each group of threads keeps
// a ring of rows in shared memory that bulk copies fill, so that the bytes in
// flight do not depend on registers.  Few rows are loaded by the threads
// here, element by element where they do not start on 16-byte boundaries.
// Rows wider than the registers hold take kernels that read x again for each
// pass (2048 x 40000: fp32 211 us, gradient 467, bfloat16 130 and 410; the copy
// rate allows 97, 145, 48 and 73).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <numeric>
#include <cstdint>

#include "../../include/gemm_f32_lm.h"
#include "device_common.cuh"
#include "launch.h"
#include "layer_norm_stream.cuh"
#include "row_common.cuh"
#include "workspace.h"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

// ---------------------------------------------------------------- forward
// G threads per row, NV vectors of VEC elements each: vector i of thread t
// holds elements (i G + t) VEC of the row.
template <class T, class WT, int VEC, int G, int NV>
__global__ void __launch_bounds__(G < 256 ? 256 : G) layer_norm_kernel(const NormArgs a) {
  constexpr int kThreads = G < 256 ? 256 : G;
  constexpr int kGroups = kThreads / G;
  __shared__ float part[2][kGroups][G / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  const long long row = static_cast<long long>(blockIdx.x) * kGroups + group;
  if (row >= a.rows) return;
  const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
  Raw<T, VEC> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = (i * G + t) * VEC;
    raw[i].zero();
    if (d < a.width && row_ok<T>(a, row * a.ldx + d, VEC, a.ldx)) raw[i].load_once(x + d);
  }
  const float inv = 1.0f / static_cast<float>(a.width);
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += raw[i].at(j);
  group_sum<1, G>(s, part[0][group], group);
  const float mean = s[0] * inv;
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * G + t) * VEC < a.width)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float c = raw[i].at(j) - mean;
        s[0] = fmaf(c, c, s[0]);
      }
  group_sum<1, G>(s, part[1][group], group);
  const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  T* const y = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = (i * G + t) * VEC;
    if (d >= a.width) break;
    float w[VEC], b[VEC], v[VEC];
    if (a.weight)
      load_cached<WT, VEC>(static_cast<const WT*>(a.weight) + d, w);
    else
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = 1.0f;
    if (a.bias)
      load_cached<WT, VEC>(static_cast<const WT*>(a.bias) + d, b);
    else
#pragma unroll
      for (int j = 0; j < VEC; ++j) b[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = fmaf((raw[i].at(j) - mean) * rstd, w[j], b[j]);
    if (row_ok<T>(a, row * a.ldo + d, VEC, a.ldo)) store_vec<T, VEC>(y + d, v);
  }
}

// Rows of any width: the row is read once for each of the three steps (from
// L2 after the first).
constexpr int kWideThreads = 1024;

template <class T, class WT>
__global__ void __launch_bounds__(kWideThreads) layer_norm_wide_kernel(const NormArgs a) {
  __shared__ float part[2][kWideThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const float inv = 1.0f / static_cast<float>(a.width);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
    float s[1] = {0.0f};
    for (unsigned d = threadIdx.x; d < static_cast<unsigned>(a.width); d += kWideThreads)
      if (row_ok<T>(a, row * a.ldx + d, 1, a.ldx)) s[0] += to_f32(x[d]);
    group_sum<1, kWideThreads>(s, part[0], 0);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
    for (unsigned d = threadIdx.x; d < static_cast<unsigned>(a.width); d += kWideThreads)
      if (row_ok<T>(a, row * a.ldx + d, 1, a.ldx)) {
        const float c = to_f32(x[d]) - mean;
        s[0] = fmaf(c, c, s[0]);
      }
    group_sum<1, kWideThreads>(s, part[1], 0);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* const y = static_cast<T*>(a.out) + row * a.ldo;
    for (unsigned d = threadIdx.x; d < static_cast<unsigned>(a.width); d += kWideThreads) {
      const float w = a.weight ? to_f32(static_cast<const WT*>(a.weight)[d]) : 1.0f;
      const float b = a.bias ? to_f32(static_cast<const WT*>(a.bias)[d]) : 0.0f;
      if (row_ok<T>(a, row * a.ldx + d, 1, a.ldx) && row_ok<T>(a, row * a.ldo + d, 1, a.ldo))
        y[d] = from_f32<T>(fmaf((to_f32(x[d]) - mean) * rstd, w, b));
    }
  }
}

// ---------------------------------------------------------------- gradient
// As the forward kernel, with a persistent grid of CTAs of kThreads threads:
// group g of CTA c takes rows c kGroups + g, then every gridDim kGroups-th.
// The next row's x and dy are loaded before the current row is reduced.
template <int G>
constexpr int kGradThreads = G < 512 ? 512 : G;

// The groups' column sums, added in group order: one row of partials per CTA.
// `cols` holds the sums of one array, kGroups G NV VEC floats.
template <class T, int VEC, int G, int NV, int THREADS>
__device__ __forceinline__ void write_columns(const NormArgs& a, float* cols, int group, int t,
                                              const float (&dw)[NV][VEC], const float (&db)[NV][VEC]) {
  constexpr int kGroups = THREADS / G, E = NV * VEC;
  if (!a.partials) return;
  float* const mine = a.partials + static_cast<size_t>(blockIdx.x) * 2 * a.width;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (kGroups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          cols[group * (G * E) + (i * G + t) * VEC + j] = which ? db[i][j] : dw[i][j];
      __syncthreads();
      for (int d = threadIdx.x; d < a.width; d += THREADS) {
        float v = cols[d];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) v += cols[g * (G * E) + d];
        mine[which * a.width + d] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int d = (i * G + t) * VEC;
        if (d < a.width)
#pragma unroll
          for (int j = 0; j < VEC; ++j) mine[which * a.width + d + j] = which ? db[i][j] : dw[i][j];
      }
    }
  }
}

template <class T, class WT, int VEC, int G, int NV>
__global__ void __launch_bounds__(kGradThreads<G>) layer_norm_grad_kernel(const NormArgs a) {
  constexpr int kThreads = kGradThreads<G>;
  constexpr int kGroups = kThreads / G;
  constexpr int E = NV * VEC;
  __shared__ float part[2][kGroups][2 * (G / 32)];
  __shared__ float cols[kGroups > 1 ? kThreads * E : 1];
  grid_launch_dependents();
  grid_dependency_wait();
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  const float inv = 1.0f / static_cast<float>(a.width);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int d = (i * G + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[i][j] = 1.0f;
      dw[i][j] = db[i][j] = 0.0f;
    }
    if (a.weight && d < a.width) load_cached<WT, VEC>(static_cast<const WT*>(a.weight) + d, w[i]);
  }
  Raw<T, VEC> xr[NV], gr[NV], xn[NV], gn[NV];
  float mean = 0.0f, rstd = 0.0f, mean_n = 0.0f, rstd_n = 0.0f;
  auto load = [&](long long row, Raw<T, VEC>(&xv)[NV], Raw<T, VEC>(&gv)[NV], float& m, float& r) {
    const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* const g = static_cast<const T*>(a.dy) + row * a.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int d = (i * G + t) * VEC;
      xv[i].zero();
      gv[i].zero();
      if (row < a.rows && d < a.width) {
        if (row_ok<T>(a, row * a.ldx + d, VEC, a.ldx)) xv[i].load_once(x + d);
        if (row_ok<T>(a, row * a.lddy + d, VEC, a.lddy)) gv[i].load_once(g + d);
      }
    }
    if (row < a.rows) {
      m = __ldg(a.mean + row);
      r = __ldg(a.rstd + row);
    }
  };
  long long row = static_cast<long long>(blockIdx.x) * kGroups + group;
  load(row, xr, gr, mean, rstd);
  int flip = 0;
  for (; row < a.rows; row += step) {
    load(row + step, xn, gn, mean_n, rstd_n);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * G + t) * VEC >= a.width) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float dy = gr[i].at(j), hat = (xr[i].at(j) - mean) * rstd;
        const float g = dy * w[i][j];
        dw[i][j] = fmaf(dy, hat, dw[i][j]);
        db[i][j] += dy;
        s[0] += g;
        s[1] = fmaf(g, hat, s[1]);
      }
    }
    if (a.out) {   // the same for every thread
      group_sum<2, G>(s, part[flip][group], group);
      flip ^= 1;
      const float c1 = s[0] * inv, c2 = s[1] * inv;
      T* const dx = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int d = (i * G + t) * VEC;
        if (d >= a.width) break;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float hat = (xr[i].at(j) - mean) * rstd;
          v[j] = rstd * (fmaf(gr[i].at(j), w[i][j], -c1) - hat * c2);
        }
        if (row_ok<T>(a, row * a.ldo + d, VEC, a.ldo)) store_vec<T, VEC>(dx + d, v);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = xn[i];
      gr[i] = gn[i];
    }
    mean = mean_n;
    rstd = rstd_n;
  }
  write_columns<T, VEC, G, NV, kThreads>(a, cols, group, t, dw, db);
}

// dweight and dbias: the sums over `count` rows of partials, 32 columns per
// CTA, row by row in 32 interleaved chains that are then added in order.
template <class WT>
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float* partials, int count,
                                                            int width, WT* dweight, WT* dbias) {
  __shared__ float sum[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, chain = threadIdx.x >> 5;
  const long long col = blockIdx.x * 32LL + lane, all = 2LL * width;
  float v = 0.0f;
  if (col < all)
    for (int r = chain; r < count; r += 32) v += __ldcg(partials + r * all + col);
  sum[chain][lane] = v;
  __syncthreads();
  if (chain == 0 && col < all) {
    float s = sum[0][lane];
#pragma unroll
    for (int c = 1; c < 32; ++c) s += sum[c][lane];
    WT* const out = col < width ? dweight : dbias;
    if (out) out[col < width ? col : col - width] = from_f32<WT>(s);
  }
}

// ---- rows of any width: the two sums of each row, then the column sums in
// bands of rows, then dx (last, so that it may overwrite x or dy).
template <class T, class WT>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_sums_kernel(const NormArgs a) {
  __shared__ float part[2][2 * (kWideThreads / 32)];
  grid_launch_dependents();
  grid_dependency_wait();
  int flip = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* const dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (unsigned d = threadIdx.x; d < static_cast<unsigned>(a.width); d += kWideThreads) {
      if (!row_ok<T>(a, row * a.ldx + d, 1, a.ldx) || !row_ok<T>(a, row * a.lddy + d, 1, a.lddy))
        continue;
      const float w = a.weight ? to_f32(static_cast<const WT*>(a.weight)[d]) : 1.0f;
      const float g = to_f32(dy[d]) * w;
      s[0] += g;
      s[1] = fmaf(g, (to_f32(x[d]) - mean) * rstd, s[1]);
    }
    group_sum<2, kWideThreads>(s, part[flip], 0);
    flip ^= 1;
    if (threadIdx.x == 0) {
      a.row_sums[2 * row] = s[0];
      a.row_sums[2 * row + 1] = s[1];
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256) norm_grad_wide_columns_kernel(const NormArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const unsigned d = blockIdx.x * 256u + threadIdx.x;
  if (d >= static_cast<unsigned>(a.width)) return;
  float dw = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    if (!row_ok<T>(a, row * a.ldx + d, 1, a.ldx) || !row_ok<T>(a, row * a.lddy + d, 1, a.lddy))
      continue;
    const float dy = to_f32(static_cast<const T*>(a.dy)[row * a.lddy + d]);
    const float hat = (to_f32(static_cast<const T*>(a.x)[row * a.ldx + d]) - a.mean[row]) * a.rstd[row];
    dw = fmaf(dy, hat, dw);
    db += dy;
  }
  float* const mine = a.partials + static_cast<size_t>(blockIdx.y) * 2 * a.width;
  mine[d] = dw;
  mine[static_cast<size_t>(a.width) + d] = db;
}

template <class T, class WT>
__global__ void __launch_bounds__(256) norm_grad_wide_dx_kernel(const NormArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const float inv = 1.0f / static_cast<float>(a.width);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float c1 = a.row_sums[2 * row] * inv, c2 = a.row_sums[2 * row + 1] * inv;
    for (unsigned d = threadIdx.x; d < static_cast<unsigned>(a.width); d += 256) {
      if (!row_ok<T>(a, row * a.ldx + d, 1, a.ldx) || !row_ok<T>(a, row * a.lddy + d, 1, a.lddy) ||
          !row_ok<T>(a, row * a.ldo + d, 1, a.ldo))
        continue;
      const float w = a.weight ? to_f32(static_cast<const WT*>(a.weight)[d]) : 1.0f;
      const float hat = (to_f32(static_cast<const T*>(a.x)[row * a.ldx + d]) - mean) * rstd;
      const float dy = to_f32(static_cast<const T*>(a.dy)[row * a.lddy + d]);
      static_cast<T*>(a.out)[row * a.ldo + d] = from_f32<T>(rstd * (fmaf(dy, w, -c1) - hat * c2));
    }
  }
}

// ---------------------------------------------------------------- host side
template <class Kernel, class... Args>
int launch(Kernel kernel, dim3 grid, int threads, cudaStream_t stream, Args... args) {
  if (launch_dependent(kernel, grid, dim3(threads), 0, stream, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

template <class T, class WT, int VEC, int G, int NV>
int launch_forward(const NormArgs& a, cudaStream_t stream) {
  constexpr int kThreads = G < 256 ? 256 : G;
  const long long ctas = (a.rows + kThreads / G - 1) / (kThreads / G);
  if (ctas > 0x7fffffffLL) return GEMM_F32_EINVAL;
  return launch(layer_norm_kernel<T, WT, VEC, G, NV>, dim3(static_cast<unsigned>(ctas)), kThreads,
                stream, a);
}

// Rows per group of a full grid from which on the streaming kernels are taken.
// From there on they are the faster ones (14592 x 1001 bfloat16 19.5 us against
// 25.9, gradient of 608 x 8192 fp32 20.9 against 29.4, 2432 x 4096 bfloat16 20.3
// against 28.8); with 1 to 3 rows per group both are bound by the host (16 to 18
// us, gradients 20 to 23; 304 x 8192 fp32 19.9 against 23.4).
constexpr int kStreamRows = 4;

// Launches a streaming kernel when the rows are many and two stages of its
// rings fit; 1 when not.
template <int G, int ARRAYS, int CTAS, void (*kernel)(NormArgs, int, int)>
int launch_stream(const NormArgs& a, bool ragged, size_t size, size_t least_smem, int device, int num_sms,
                  int* parts, cudaStream_t stream) {
  constexpr int kGroups = stream_threads(G) / G;
  // a multiple of 8 groups on ragged rows: of one start each
  constexpr int kWhole = 8 / std::gcd(8, kGroups);
  static std::atomic<int> resident[64];    // of this kernel: CTAs or clusters at a time, per device
  int most = resident[device % 64].load();
  if (most == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kStreamBytes)) != cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    most = num_sms;
    if (CTAS > 1) {   // as many as run at once (36 of four CTAs: 2048 x 32768 bfloat16 96 us, 167 with 38)
      cudaLaunchConfig_t config = {};
      config.gridDim = dim3(num_sms / CTAS * CTAS);
      config.blockDim = dim3(stream_threads(G));
      config.dynamicSmemBytes = kStreamBytes;
      if (cudaOccupancyMaxActiveClusters(&most, kernel, &config) != cudaSuccess || most < 1) {
        (void)cudaGetLastError();
        return GEMM_F32_ELAUNCH;
      }
    }
    resident[device % 64].store(most);
  }
  const int units = ragged ? most / kWhole * kWhole : most, grid = units * CTAS;
  // of a shared row: whole 16-byte blocks, of which a ragged row may take one more than its elements fill
  const long long blocks = a.width + (ragged ? 16 / static_cast<long long>(size) - 1 : 0);
  const int slice = CTAS == 1 ? a.width : static_cast<int>(((blocks + CTAS - 1) / CTAS + 7) / 8 * 8);
  const size_t row = ring_row_bytes(slice, size, ragged) * ARRAYS;
  const int stages = static_cast<int>(std::min<size_t>(kMostStages, kStreamBytes / (kGroups * (row + 8))));
  if (a.rows < static_cast<long long>(kStreamRows) * units * kGroups || stages < 2 || units == 0) return 1;
  const size_t smem = std::max(least_smem, kGroups * stages * (row + 8));
  *parts = units;
  if (launch_dependent(kernel, dim3(grid), dim3(stream_threads(G)), smem, stream, a, stages, slice) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

// How the rows of a call's matrices lie: all on 16-byte boundaries, or row by
// row equally far from one in every matrix, or neither (which the streaming
// kernels do not take).
enum class Rows { kVectors, kRagged, kUneven };

// E elements of a row per thread.
template <class T, class WT, int G, int E>
int stream_forward(const NormArgs& a, Rows rows, int device, int num_sms, cudaStream_t stream) {
  int parts;
  return rows == Rows::kVectors ? launch_stream<G, 1, 1, layer_norm_stream_kernel<T, WT, G, E / 2, false>>(
                       a, false, sizeof(T), 0, device, num_sms, &parts, stream)
                 : launch_stream<G, 1, 1, layer_norm_stream_kernel<T, WT, G, E / 2, true>>(
                       a, true, sizeof(T), 0, device, num_sms, &parts, stream);
}

template <class T, class WT, int G, int E, int CTAS = 1>
int stream_grad(NormArgs a, Rows rows, float* scratch, int device, int num_sms, int* parts,
                cudaStream_t stream) {
  a.partials = scratch;
  constexpr size_t kColumns = sizeof(float) * stream_threads(G) * E;
  return rows == Rows::kVectors ? launch_stream<G, 2, CTAS, layer_norm_grad_stream_kernel<T, WT, G, E / 2, false, CTAS>>(
                       a, false, sizeof(T), kColumns, device, num_sms, parts, stream)
                 : launch_stream<G, 2, CTAS, layer_norm_grad_stream_kernel<T, WT, G, E / 2, true, CTAS>>(
                       a, true, sizeof(T), kColumns, device, num_sms, parts, stream);
}

// The narrowest group of threads whose registers hold the row: up to 4
// vectors a thread, or 8 elements where they are read one by one.
template <class T, class WT>
int forward(const NormArgs& a, Rows rows, int device, int num_sms, cudaStream_t stream, const char** kernel) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool vectors = rows == Rows::kVectors;
  const int n = vectors ? (a.width - 1) / V + 1 : a.width;
  if (rows != Rows::kUneven) {
    const long long e = a.width + (vectors ? 0LL : V - 1LL);   // a row's start may take part of a vector
    const int rc = e <= 256     ? stream_forward<T, WT, 32, 8>(a, rows, device, num_sms, stream)
                   : e <= 512   ? stream_forward<T, WT, 32, 16>(a, rows, device, num_sms, stream)
                   : e <= 768   ? stream_forward<T, WT, 32, 24>(a, rows, device, num_sms, stream)
                   : e <= 1024  ? stream_forward<T, WT, 32, 32>(a, rows, device, num_sms, stream)
                   : e <= 1536  ? stream_forward<T, WT, 64, 24>(a, rows, device, num_sms, stream)
                   : e <= 2048  ? stream_forward<T, WT, 64, 32>(a, rows, device, num_sms, stream)
                   : e <= 3072  ? stream_forward<T, WT, 128, 24>(a, rows, device, num_sms, stream)
                   : e <= 4096  ? stream_forward<T, WT, 128, 32>(a, rows, device, num_sms, stream)
                   : e <= 6144  ? stream_forward<T, WT, 256, 24>(a, rows, device, num_sms, stream)
                   : e <= 8192  ? stream_forward<T, WT, 256, 32>(a, rows, device, num_sms, stream)
                   : e <= 12288 ? stream_forward<T, WT, 512, 24>(a, rows, device, num_sms, stream)
                   : e <= 16384 ? stream_forward<T, WT, 512, 32>(a, rows, device, num_sms, stream)
                                : 1;
    if (rc != 1) {
      *kernel = "layer_norm_stream_kernel";
      return rc;
    }
  }
  *kernel = "layer_norm_kernel";
  if (vectors) {
    if (n <= 32) return launch_forward<T, WT, V, 32, 1>(a, stream);
    if (n <= 64) return launch_forward<T, WT, V, 32, 2>(a, stream);
    if (n <= 128) return launch_forward<T, WT, V, 32, 4>(a, stream);
    if (n <= 256) return launch_forward<T, WT, V, 128, 2>(a, stream);
    if (n <= 512) return launch_forward<T, WT, V, 256, 2>(a, stream);
    if (n <= 1024) return launch_forward<T, WT, V, 256, 4>(a, stream);
    if (n <= 2048) return launch_forward<T, WT, V, 512, 4>(a, stream);
    if (n <= 4096) return launch_forward<T, WT, V, 1024, 4>(a, stream);
  } else {
    if (n <= 256) return launch_forward<T, WT, 1, 32, 8>(a, stream);
    if (n <= 1024) return launch_forward<T, WT, 1, 128, 8>(a, stream);
    if (n <= 2048) return launch_forward<T, WT, 1, 256, 8>(a, stream);
    if (n <= 4096) return launch_forward<T, WT, 1, 512, 8>(a, stream);
    if (n <= 8192) return launch_forward<T, WT, 1, 1024, 8>(a, stream);
  }
  const unsigned ctas = static_cast<unsigned>(std::min<long long>(a.rows, 2LL * num_sms));
  return launch(layer_norm_wide_kernel<T, WT>, dim3(ctas), kWideThreads, stream, a);
}

constexpr int kWideBands = 64;

template <class T, class WT, int VEC, int G, int NV>
int launch_grad(NormArgs a, float* scratch, int num_sms, int* ctas, cudaStream_t stream) {
  constexpr int kThreads = kGradThreads<G>;
  constexpr int kGroups = kThreads / G;
  const long long most = (a.rows + kGroups - 1) / kGroups;
  *ctas = static_cast<int>(std::min<long long>(most, 2LL * num_sms));
  a.partials = scratch;
  return launch(layer_norm_grad_kernel<T, WT, VEC, G, NV>, dim3(*ctas), kThreads, stream, a);
}

template <class T, class WT>
int grad(NormArgs a, Rows rows, void* dweight, void* dbias, int device, int num_sms,
         cudaStream_t stream, int* launches, const char** kernel) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const bool columns = dweight || dbias, vectors = rows == Rows::kVectors;
  const int n = vectors ? (a.width - 1) / V + 1 : a.width;
  // vectors (elements where unaligned) that the widest register kernel holds
  const bool wide = n > (vectors ? 16384 / V : 8192);
  const long long bands = std::min<long long>(a.rows, 2LL * num_sms);   // at most, in any kernel
  const size_t part_floats = columns ? static_cast<size_t>(bands) * 2 * a.width : 0;
  const size_t sums_floats = wide ? 2 * static_cast<size_t>(a.rows) : 0;
  float* scratch = nullptr;
  if (part_floats + sums_floats) {
    scratch = static_cast<float*>(
        acquire_scratch(device, stream, (part_floats + sums_floats) * sizeof(float)));
    if (!scratch) return GEMM_F32_ESCRATCH;
  }
  float* const parts = columns ? scratch : nullptr;
  int ctas = 0, rc;
  *kernel = "layer_norm_grad_kernel";
  if (a.rows == 0) {
    *kernel = "norm_columns_kernel";
    rc = GEMM_F32_OK;
  } else {
    const long long e = a.width + (vectors ? 0LL : V - 1LL);
    rc = rows == Rows::kUneven ? 1
         : e <= 256   ? stream_grad<T, WT, 32, 8>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 512   ? stream_grad<T, WT, 32, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 1024  ? stream_grad<T, WT, 64, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 1536  ? stream_grad<T, WT, 96, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 2048  ? stream_grad<T, WT, 128, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 3072  ? stream_grad<T, WT, 192, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 4096  ? stream_grad<T, WT, 256, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 6144  ? stream_grad<T, WT, 384, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 8192  ? stream_grad<T, WT, 512, 16>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 12288 ? stream_grad<T, WT, 384, 16, 2>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 16384 ? stream_grad<T, WT, 512, 16, 2>(a, rows, parts, device, num_sms, &ctas, stream)
         : e <= 32768 ? stream_grad<T, WT, 512, 16, 4>(a, rows, parts, device, num_sms, &ctas, stream)
                      : 1;
    if (rc != 1) {
      *kernel = "layer_norm_grad_stream_kernel";
      ++*launches;
    }
  }
  if (rc == 1 && !wide) {
    if (vectors && V == 8) {
      if (n <= 32) rc = launch_grad<T, WT, V, 32, 1>(a, parts, num_sms, &ctas, stream);
      else if (n <= 64) rc = launch_grad<T, WT, V, 32, 2>(a, parts, num_sms, &ctas, stream);
      else if (n <= 128) rc = launch_grad<T, WT, V, 128, 1>(a, parts, num_sms, &ctas, stream);
      else if (n <= 256) rc = launch_grad<T, WT, V, 256, 1>(a, parts, num_sms, &ctas, stream);
      else if (n <= 512) rc = launch_grad<T, WT, V, 512, 1>(a, parts, num_sms, &ctas, stream);
      else if (n <= 1024) rc = launch_grad<T, WT, V, 1024, 1>(a, parts, num_sms, &ctas, stream);
      else rc = launch_grad<T, WT, V, 1024, 2>(a, parts, num_sms, &ctas, stream);
    } else if (vectors) {
      if (n <= 32) rc = launch_grad<T, WT, V, 32, 1>(a, parts, num_sms, &ctas, stream);
      else if (n <= 64) rc = launch_grad<T, WT, V, 32, 2>(a, parts, num_sms, &ctas, stream);
      else if (n <= 128) rc = launch_grad<T, WT, V, 32, 4>(a, parts, num_sms, &ctas, stream);
      else if (n <= 256) rc = launch_grad<T, WT, V, 128, 2>(a, parts, num_sms, &ctas, stream);
      else if (n <= 512) rc = launch_grad<T, WT, V, 256, 2>(a, parts, num_sms, &ctas, stream);
      else if (n <= 1024) rc = launch_grad<T, WT, V, 512, 2>(a, parts, num_sms, &ctas, stream);
      else if (n <= 2048) rc = launch_grad<T, WT, V, 1024, 2>(a, parts, num_sms, &ctas, stream);
      else rc = launch_grad<T, WT, V, 1024, 4>(a, parts, num_sms, &ctas, stream);
    } else {
      if (n <= 256) rc = launch_grad<T, WT, 1, 32, 8>(a, parts, num_sms, &ctas, stream);
      else if (n <= 1024) rc = launch_grad<T, WT, 1, 128, 8>(a, parts, num_sms, &ctas, stream);
      else if (n <= 2048) rc = launch_grad<T, WT, 1, 256, 8>(a, parts, num_sms, &ctas, stream);
      else if (n <= 4096) rc = launch_grad<T, WT, 1, 512, 8>(a, parts, num_sms, &ctas, stream);
      else rc = launch_grad<T, WT, 1, 1024, 8>(a, parts, num_sms, &ctas, stream);
    }
    ++*launches;
  } else if (rc == 1) {
    const unsigned grid = static_cast<unsigned>(std::min<long long>(a.rows, 2LL * num_sms));
    a.row_sums = scratch + part_floats;
    rc = GEMM_F32_OK;
    if (a.out) {
      rc = launch(norm_grad_wide_sums_kernel<T, WT>, dim3(grid), kWideThreads, stream, a);
      ++*launches;
    }
    if (rc == GEMM_F32_OK && columns) {
      ctas = static_cast<int>(std::min<long long>(a.rows, kWideBands));
      a.partials = parts;
      rc = launch(norm_grad_wide_columns_kernel<T>,
                  dim3((a.width + 255u) / 256u, static_cast<unsigned>(ctas)), 256, stream, a);
      ++*launches;
    }
    if (rc == GEMM_F32_OK && a.out) {
      rc = launch(norm_grad_wide_dx_kernel<T, WT>, dim3(4 * grid), 256, stream, a);
      ++*launches;
    }
  }
  if (rc == GEMM_F32_OK && columns) {
    const unsigned grid = static_cast<unsigned>((2LL * a.width + 31) / 32);
    rc = launch(norm_columns_kernel<WT>, dim3(grid), 1024, stream,
                static_cast<const float*>(parts), ctas, a.width, static_cast<WT*>(dweight),
                static_cast<WT*>(dbias));
    ++*launches;
  }
  return rc;
}

size_t type_size(int type) { return type == GEMM_F32_TYPE_F32 ? 4 : 2; }

// Checks shared by both entry points.
bool common_ok(int type, int weight_type, long long rows, int width) {
  return (type == GEMM_F32_TYPE_F32 || type == GEMM_F32_TYPE_BF16) &&
         (weight_type == GEMM_F32_TYPE_F32 || weight_type == type) && rows >= 0 && width >= 1;
}

bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// A matrix operand: present, aligned to its element, stride at least a row.
bool matrix_ok(const void* p, long long ld, int width, size_t size) {
  return p && aligned_to(p, size) && ld >= width;
}

size_t matrix_bytes(long long rows, int width, long long ld, size_t size) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * ld + width) * size : 0;
}

// Rows of the matrix start on 16-byte boundaries and hold whole vectors.
bool vector_rows(const void* p, long long ld, int width, size_t size) {
  return aligned_to(p, 16) && ld * size % 16 == 0 && width * size % 16 == 0;
}

// Row by row as far from a 16-byte boundary as in the other matrix.
bool alike(const void* p, long long ldp, const void* q, long long ldq, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) % 16 == 0 &&
         (ldp - ldq) * static_cast<long long>(size) % 16 == 0;
}

// An output that is an input matrix itself, or apart from it.
bool same_or_apart(const void* out, long long ldo, const void* in, long long ldi, long long rows,
                   int width, size_t size) {
  if (out == in && ldo == ldi) return true;
  return !ranges_overlap(out, matrix_bytes(rows, width, ldo, size), in,
                         matrix_bytes(rows, width, ldi, size));
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" int gemm_f32_layer_norm(int type, int weight_type, long long rows, int width,
                                   const void* x, long long ldx, const void* weight,
                                   const void* bias, float eps, void* y, long long ldy,
                                   float* mean, float* rstd, gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!common_ok(type, weight_type, rows, width)) return GEMM_F32_EINVAL;
  if (!std::isfinite(eps) || eps < 0.0f) return GEMM_F32_EINVAL;
  if (rows == 0) return GEMM_F32_OK;
  const size_t es = type_size(type), ws = type_size(weight_type);
  if (!matrix_ok(x, ldx, width, es) || !matrix_ok(y, ldy, width, es)) return GEMM_F32_EINVAL;
  if (!aligned_to(weight, ws) || !aligned_to(bias, ws) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return GEMM_F32_EINVAL;
  if (!same_or_apart(y, ldy, x, ldx, rows, width, es)) return GEMM_F32_EINVAL;
  NormArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.rows = rows;
  a.width = width;
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.out = y;
  a.ldo = ldy;
  a.mean = mean;
  a.rstd = rstd;
  const bool vectors = vector_rows(x, ldx, width, es) && vector_rows(y, ldy, width, es) &&
                       aligned_to(weight, 16) && aligned_to(bias, 16);
  const Rows how = vectors                       ? Rows::kVectors
                   : alike(x, ldx, y, ldy, es)   ? Rows::kRagged
                                                 : Rows::kUneven;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  int rc;
  const char* kernel = "none";
  if (type == GEMM_F32_TYPE_F32)
    rc = forward<float, float>(a, how, device, num_sms, stream, &kernel);
  else if (weight_type == GEMM_F32_TYPE_F32)
    rc = forward<bf16, float>(a, how, device, num_sms, stream, &kernel);
  else
    rc = forward<bf16, bf16>(a, how, device, num_sms, stream, &kernel);
  if (rc == GEMM_F32_OK) note_launches(1, kernel);
  return rc;
}

extern "C" int gemm_f32_layer_norm_grad(int type, int weight_type, long long rows, int width,
                                        const void* dy, long long lddy, const void* x,
                                        long long ldx, const void* weight, const float* mean,
                                        const float* rstd, void* dx, long long lddx,
                                        void* dweight, void* dbias,
                                        gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!common_ok(type, weight_type, rows, width)) return GEMM_F32_EINVAL;
  const size_t es = type_size(type), ws = type_size(weight_type);
  if (!aligned_to(weight, ws) || !aligned_to(dweight, ws) || !aligned_to(dbias, ws))
    return GEMM_F32_EINVAL;
  if (rows > 0) {
    if (!matrix_ok(dy, lddy, width, es) || !matrix_ok(x, ldx, width, es)) return GEMM_F32_EINVAL;
    if (!mean || !rstd || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return GEMM_F32_EINVAL;
    if (dx) {
      if (!matrix_ok(dx, lddx, width, es)) return GEMM_F32_EINVAL;
      if (!same_or_apart(dx, lddx, dy, lddy, rows, width, es) ||
          !same_or_apart(dx, lddx, x, ldx, rows, width, es))
        return GEMM_F32_EINVAL;
    }
  }
  const bool columns = dweight || dbias;
  if (!columns && (rows == 0 || !dx)) return GEMM_F32_OK;
  NormArgs a = {};
  int device = 0, num_sms = 0;
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  a.rows = rows;
  a.width = width;
  a.x = x;
  a.ldx = ldx;
  a.dy = dy;
  a.lddy = lddy;
  a.weight = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.out = dx;
  a.ldo = lddx;
  const bool vectors = vector_rows(x, ldx, width, es) && vector_rows(dy, lddy, width, es) &&
                       (!dx || vector_rows(dx, lddx, width, es)) && aligned_to(weight, 16);
  const Rows how = vectors ? Rows::kVectors
                   : alike(x, ldx, dy, lddy, es) && (!dx || alike(x, ldx, dx, lddx, es)) ? Rows::kRagged
                                                                                        : Rows::kUneven;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  int rc, launches = 0;
  const char* kernel = "none";
  const WorkspaceCall call;
  if (type == GEMM_F32_TYPE_F32)
    rc = grad<float, float>(a, how, dweight, dbias, device, num_sms, stream, &launches, &kernel);
  else if (weight_type == GEMM_F32_TYPE_F32)
    rc = grad<bf16, float>(a, how, dweight, dbias, device, num_sms, stream, &launches, &kernel);
  else
    rc = grad<bf16, bf16>(a, how, dweight, dbias, device, num_sms, stream, &launches, &kernel);
  if (rc == GEMM_F32_OK) note_launches(launches, kernel);
  return rc;
}
