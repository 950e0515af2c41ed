// Device-side helpers of the row operators (layer norm, vocabulary loss):
// element types, vector loads and stores, and reductions over the threads
// that share a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "launch.h"

namespace gemm_f32_dev {
using gemm_f32_impl::kSiteTarget;
using gemm_f32_impl::LossTargets;

// Sites of the checked build, after those of device_common.cuh.
constexpr unsigned kSiteBoundsRows = 21;      // a row of a layer norm or a loss outside its matrix
constexpr unsigned kSiteBoundsScratch = 22;   // a layer norm's or a loss's scratch outside its part

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N elements of T held as raw bits, so that a load can be in flight while
// nothing of it is converted yet.
template <class T, int N>
struct Raw {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];

  // p is aligned to min(16, kBytes) bytes.  Read once: streamed past L1.
  __device__ __forceinline__ void load_once(const T* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = q.x;
        w[4 * i + 1] = q.y;
        w[4 * i + 2] = q.z;
        w[4 * i + 3] = q.w;
      }
    } else {
      static_assert(N == 1, "vectors are 16 bytes");
      if constexpr (sizeof(T) == 4)
        w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
      else
        w[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
  }
};

// Two fp32 values in one 64-bit register: the packed operations do both in
// one instruction, each rounded to nearest as by itself.
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void unpair(Pair p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ float sum_of(Pair p) {
  float a, b;
  unpair(p, a, b);
  return a + b;
}

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Powers of the logits z of a tile relative to its maximum m are
// 2^((z - m) log2 e).  z - m first: it is exact near the maximum, whatever its
// size.  A product z log2 e - m log2 e by fma is off by half a last place of
// m log2 e, which is whole powers of 2 for logits of 10^7 (masks of -10^10 gave
// infinite sums), and it overflows from 2.36e38 on.
constexpr float kLog2e = 1.4426950408889634f;

// What the powers are taken relative to: of a tile with nothing above -inf any
// finite value gives powers of 0.
__device__ __forceinline__ float reference(float top) { return top == -INFINITY ? 0.0f : top; }

// 16 bytes as pairs: 2 of fp32, 4 of bfloat16.
template <class T>
__device__ __forceinline__ void pairs_of(const uint4& q, Pair (&v)[8 / sizeof(T)]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
    v[0] = pair_of(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = pair_of(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
}

// N consecutive elements as fp32, through the cache (weights that every row reads).
template <class T, int N>
__device__ __forceinline__ void load_cached(const T* p, float (&v)[N]) {
  if constexpr (N * sizeof(T) >= 16) {
    Raw<T, N> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(N * sizeof(T) / 16); ++i) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = q.x;
      r.w[4 * i + 1] = q.y;
      r.w[4 * i + 2] = q.z;
      r.w[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = r.at(i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(p[i]);
  }
}

template <class T, int N>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    p[0] = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    static_assert(N % 4 == 0, "16-byte stores");
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    static_assert(N % 8 == 0, "16-byte stores");
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      reinterpret_cast<uint4*>(p)[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

template <class T>
__device__ __forceinline__ void store_pairs(T* p, const Pair (&v)[8 / sizeof(T)]) {
  constexpr int N = 8 / sizeof(T);
  float f[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) unpair(v[i], f[2 * i], f[2 * i + 1]);
  store_vec<T, 2 * N>(p, f);
}

// The label of a row of a loss: its target, or -1 where the row does not
// count (its target is the ignored one, or outside the vocabulary).
__device__ __forceinline__ int label_at(const LossTargets& t, long long row) {
  const long long y = t.bits == 64 ? __ldg(static_cast<const long long*>(t.p) + row)
                                   : __ldg(static_cast<const int*>(t.p) + row);
  return y != t.ignore && y >= 0 && y < t.vocab ? static_cast<int>(y) : -1;
}

template <int N>
__device__ __forceinline__ void warp_sum(float (&v)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

// Sums of N values over the G threads that share a row (G a multiple of 32;
// every thread gets the sums).  `part` is the group's own shared memory of
// N * G / 32 floats, which must not be written again before a barrier of the
// group has passed: callers alternate two of them.  Groups of more than one
// warp meet at the named barrier 1 + group.
template <int N, int G>
__device__ __forceinline__ void group_sum(float (&v)[N], float* part, int group) {
  static_assert(G % 32 == 0, "whole warps");
  constexpr int W = G / 32;
  warp_sum<N>(v);
  if constexpr (W > 1) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x % G) >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[i * W + warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(G) : "memory");
    if constexpr (W <= 8) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = part[i * W];
#pragma unroll
        for (int j = 1; j < W; ++j) v[i] += part[i * W + j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = lane < W ? part[i * W + lane] : 0.0f;
      warp_sum<N>(v);
    }
  }
}

}  // namespace gemm_f32_dev
