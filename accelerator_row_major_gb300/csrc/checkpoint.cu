// Activations kept in 8 bits (saved_rows.cuh), brought back, and the weight
// gradient of a product whose input was kept (sm_103a).
//
// Both conversions are bound by memory traffic: 3 bytes an element in bfloat16,
// 5 in fp32, and a byte per 32 elements.  A warp takes 256 columns of a row at
// a time, some such pieces in flight, a lane 8 columns (a block is four lanes).
// Codes start on 16-byte boundaries; rows of the matrix that do not are moved
// in 16-byte blocks all the same, and shifted against the codes in registers.
//
// The weight gradient dw = dy^T x is a product on the tensor cores
// (half_gemm.cu) that reads both operands as they are stored.  e4m3 codes
// times powers of two are bfloat16 numbers, so x is brought back into scratch
// without a rounding; an fp32 dy goes in three parts, against an x that is
// one: three products where fp32 operands take six.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "../../include/gemm_f32_block.h"
#include "device_common.cuh"
#include "half_gemm.h"
#include "launch.h"
#include "row_common.cuh"
#include "saved_rows.cuh"
#include "workspace.h"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

using bf16 = __nv_bfloat16;

constexpr int kConvertThreads = 256;
constexpr int kPiece = 256;              // columns of a warp's piece

// Pieces in flight per warp.  Keeping other rows than bfloat16 ones on
// boundaries, more warps are worth more than more pieces a warp (65536 x 1024
// fp32 52 us with two against 56, bfloat16 44 against 42; 65536 x 1001 bfloat16
// 63 against 72, fp32 72 against 93).
constexpr int kRestoreFlight = 4;
template <class T, bool VEC>
constexpr int keep_flight() {
  return sizeof(T) == 2 && VEC ? 4 : 2;
}

struct ConvertArgs {
  long long rows;
  int width;                             // columns of x; restoring: columns to write
  const void* x;                         // keeping: read; restoring: null
  void* out;                             // restoring: written
  long long ld;                          // of x or out, elements
  uint8_t* codes;
  long long ld_codes;
  uint8_t* exponents;
  long long ld_exponents;
  int pieces;                            // per row
  unsigned* err;
};

// The pieces of one warp: `flight` side by side at a time, the CTA's warps side
// by side, and on by a grid of them.  One division at the start.
struct Pieces {
  long long row, d_row;
  int piece, per_row, d_piece;

  __device__ __forceinline__ Pieces(int per, int flight, unsigned cta, unsigned ctas) : per_row(per) {
    constexpr int kWarps = kConvertThreads / 32;
    const long long first = (cta * static_cast<long long>(kWarps) + (threadIdx.x >> 5)) * flight;
    const long long skip = (ctas * static_cast<long long>(kWarps) - 1) * flight;
    row = first / per;
    piece = static_cast<int>(first - row * per);
    d_row = skip / per;
    d_piece = static_cast<int>(skip - d_row * per);
  }
  __device__ __forceinline__ void next() {
    if (++piece == per_row) {
      piece = 0;
      ++row;
    }
  }
  __device__ __forceinline__ void next_grid() {
    row += d_row;
    piece += d_piece;
    if (piece >= per_row) {
      piece -= per_row;
      ++row;
    }
  }
};

template <class T>
__device__ __forceinline__ bool x_ok(const ConvertArgs& a, long long row, int last) {
  return GEMM_IN_EXTENT(row * a.ld + last, stored_extent(a.rows, a.width, a.ld), a.err, kSiteBoundsRows);
}
__device__ __forceinline__ bool codes_ok(const ConvertArgs& a, long long row, int last) {
  return GEMM_IN_EXTENT(row * a.ld_codes + last, a.rows * a.ld_codes, a.err, kSiteBoundsRows) &&
         GEMM_IN_EXTENT(row * a.ld_exponents + last / kSavedBlock, a.rows * a.ld_exponents, a.err, kSiteBoundsRows);
}

// ---------------------------------------------------------------- keeping
// 8 elements of a row that starts `off` bytes above a 16-byte boundary, from
// the whole blocks that they lie in: the lane's own ones and the first of the
// next lane's (the last lane loads it), shifted.  The same off for all lanes.
template <class T>
__device__ __forceinline__ void load_shifted(const T* p, uint32_t off, Raw<T, 8>& x) {
  constexpr int kWords = Raw<T, 8>::kWords;
  const int lane = threadIdx.x & 31;
  const uint4* const from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15});
  uint32_t w[kWords + 4];
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i) {
    const uint4 q = __ldcs(from + i);
    w[4 * i] = q.x;
    w[4 * i + 1] = q.y;
    w[4 * i + 2] = q.z;
    w[4 * i + 3] = q.w;
  }
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (lane == 31) q = __ldcs(from + kWords / 4);
  const uint32_t last[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
    w[kWords + i] = lane == 31 ? last[i] : next;
  }
  const auto take = [&](auto words) {
    constexpr int kFrom = decltype(words)::value;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      x.w[i] = sizeof(T) == 2 ? __funnelshift_r(w[i + kFrom], w[min(i + kFrom + 1, kWords + 3)], off % 4 * 8) : w[i + kFrom];
  };
  switch (off / 4) {
    case 0: take(std::integral_constant<int, 0>{}); break;
    case 1: take(std::integral_constant<int, 1>{}); break;
    case 2: take(std::integral_constant<int, 2>{}); break;
    default: take(std::integral_constant<int, 3>{}); break;
  }
}

// VEC: rows on 16-byte boundaries of whole vectors; else rows that start
// anywhere, shifted into place (by single elements where the blocks around
// them are not all the matrix's: at its two ends).
template <class T, bool VEC>
__global__ void __launch_bounds__(kConvertThreads, keep_flight<T, VEC>() == 2 ? 6 : 4)
    checkpoint_kernel(const ConvertArgs a) {
  constexpr int kFlight = keep_flight<T, VEC>();
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  for (Pieces at(a.pieces, kFlight, blockIdx.x, gridDim.x); at.row < a.rows; at.next_grid()) {
    // all pieces' loads first
    long long row[kFlight];
    int col[kFlight];                    // of the lane's first element
    Raw<T, 8> x[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      row[f] = at.row;
      const int col0 = at.piece * kPiece;
      col[f] = col0 + lane * 8;
      at.next();
      x[f].zero();
      if (row[f] >= a.rows) continue;    // the warp's
      const T* const p = static_cast<const T*>(a.x) + row[f] * a.ld + col[f];
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
          Raw<T, V> q;
          q.zero();
          if (col[f] + i * V < a.width && x_ok<T>(a, row[f], col[f] + i * V + V - 1)) q.load_once(p + i * V);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[f].w[4 * i + j] = q.w[j];
        }
      } else {
        // bytes from the matrix's first to this piece's blocks and to their end
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        const long long before = (row[f] * a.ld + col0) * static_cast<long long>(sizeof(T)) - off;
        const long long end = before + kPiece * static_cast<long long>(sizeof(T)) + 16;
        const bool inside = before >= 0 && end <= static_cast<long long>(stored_extent(a.rows, a.width, a.ld) * sizeof(T));
        if (inside) {
          load_shifted<T>(p, off, x[f]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            Raw<T, 1> e;
            e.zero();
            if (col[f] + j < a.width && x_ok<T>(a, row[f], col[f] + j)) e.load_once(p + j);
            if constexpr (sizeof(T) == 4)
              x[f].w[j] = e.w[0];
            else
              x[f].w[j / 2] |= e.w[0] << (16 * (j & 1));
          }
        }
        if (col0 + kPiece > a.width) {   // the row's last piece: nothing behind its end
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col[f] + j >= a.width) x[f].w[sizeof(T) == 4 ? j : j / 2] &= sizeof(T) == 4 ? 0u : (j & 1 ? 0xFFFFu : 0xFFFF0000u);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (row[f] >= a.rows) break;
      const int c = col[f];
      uint32_t top = largest_bits(x[f]);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const bool odd = __any_sync(0xFFFFFFFFu, top >= kOddBits);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x[f].at(j);
      if (odd) {                         // perhaps not finite
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, finite_bits(v[j]));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      }
      const uint32_t e = block_exponent(top);
      const float by = inverse_of(e);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float q, r;
        unpair(mul2(pair_of(v[2 * j], v[2 * j + 1]), pair_of(by, by)), q, r);
        w[j] = odd ? codes_of(q, r, e == kLargestExponent ? 240.0f : 448.0f) : finite_codes(q, r);
      }
      if (c - lane % 4 * 8 >= a.width || !codes_ok(a, row[f], c + 7)) continue;   // no such block
      *reinterpret_cast<uint2*>(a.codes + row[f] * a.ld_codes + c) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      if (lane % 4 == 0) a.exponents[row[f] * a.ld_exponents + c / kSavedBlock] = static_cast<uint8_t>(e);
    }
  }
}

// ---------------------------------------------------------------- bringing back
// VEC: rows on 16-byte boundaries; a row's last vector may reach past its last
// column, where its codes are 0 (scratch rows).  Else a lane has the 8
// elements of whole 16-byte blocks of the output, `above` elements before the
// 8 of its codes, which it takes with those before (the lane's before).
template <class T, bool VEC>
__device__ __forceinline__ void restore_rows(const ConvertArgs& a, unsigned cta, unsigned ctas) {
  constexpr int kFlight = kRestoreFlight;
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  for (Pieces at(a.pieces, kFlight, cta, ctas); at.row < a.rows; at.next_grid()) {
    long long row[kFlight];
    int col[kFlight];                    // of the lane's codes
    uint2 w[kFlight], before[kFlight];
    uint8_t e[kFlight], e_before[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      row[f] = at.row;
      col[f] = at.piece * kPiece + lane * 8;
      at.next();
      w[f] = before[f] = make_uint2(0u, 0u);
      e[f] = e_before[f] = 1;
      if (row[f] >= a.rows) continue;
      const uint8_t* const codes = a.codes + row[f] * a.ld_codes;
      const uint8_t* const exponents = a.exponents + row[f] * a.ld_exponents;
      const int c = col[f];
      if (c < a.width && codes_ok(a, row[f], c + 7)) {
        w[f] = __ldcs(reinterpret_cast<const uint2*>(codes + c));
        e[f] = __ldg(exponents + c / kSavedBlock);
      }
      if (!VEC && c > 0 && c - 8 < a.width && codes_ok(a, row[f], c - 1)) {
        if (lane == 0) before[f] = __ldcs(reinterpret_cast<const uint2*>(codes + c - 8));
        e_before[f] = __ldg(exponents + (c - 8) / kSavedBlock);
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (row[f] >= a.rows) break;
      T* const out = static_cast<T*>(a.out) + row[f] * a.ld;
      int c = col[f];
      float v[8];
      if constexpr (VEC) {
        const float by = power_of(e[f]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = values_of(((j < 2 ? w[f].x : w[f].y) >> (16 * (j & 1))) & 0xFFFFu);
          v[2 * j] = p.x * by;
          v[2 * j + 1] = p.y * by;
        }
      } else {
        const int above = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T));
        const uint2 left = make_uint2(__shfl_up_sync(0xFFFFFFFFu, w[f].x, 1), __shfl_up_sync(0xFFFFFFFFu, w[f].y, 1));
        if (lane > 0) before[f] = left;
        // bytes 8 - above .. 15 - above of the 16
        const unsigned long long lo = static_cast<unsigned long long>(before[f].y) << 32 | before[f].x;
        const unsigned long long hi = static_cast<unsigned long long>(w[f].y) << 32 | w[f].x;
        const unsigned long long q = above ? lo >> (8 * (8 - above)) | hi << (8 * above) : hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = values_of(static_cast<uint32_t>(q >> (16 * j)) & 0xFFFFu);
          v[2 * j] = p.x * power_of(2 * j < above ? e_before[f] : e[f]);
          v[2 * j + 1] = p.y * power_of(2 * j + 1 < above ? e_before[f] : e[f]);
        }
        c -= above;
      }
#pragma unroll
      for (int i = 0; i < 8 / V; ++i) {
        float part[V];
#pragma unroll
        for (int j = 0; j < V; ++j) part[j] = v[i * V + j];
        const int first = c + i * V;
        if (VEC ? first < a.width : first >= 0 && first + V <= a.width) {
          if (x_ok<T>(a, row[f], first + V - 1)) store_vec<T, V>(out + first, part);
        } else if (!VEC) {               // the row's ends
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (first + j >= 0 && first + j < a.width && x_ok<T>(a, row[f], first + j)) out[first + j] = from_f32<T>(part[j]);
        }
      }
    }
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kConvertThreads) restore_kernel(const ConvertArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  restore_rows<T, VEC>(a, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- operands of the weight gradient
// dy as the tensor cores read it: bfloat16 copied into rows on 16-byte
// boundaries, or fp32 in three planes of bfloat16.  hi is the value truncated
// (so that it never overflows), mid and lo round what is left to nearest; the
// rest is below 2^-25 of the value.
struct SplitArgs {
  const void* src;
  bf16* dst;
  long long ld, ld_dst, plane, vectors;  // vectors of 8 in all rows of dst
  int rows, cols, aligned;
};

template <class T>
__device__ __forceinline__ void split_rows(const SplitArgs& m, unsigned cta, unsigned ctas, unsigned* err) {
  const int per_row = static_cast<int>(m.ld_dst / 8);
  for (long long i = cta * static_cast<long long>(kConvertThreads) + threadIdx.x; i < m.vectors;
       i += ctas * static_cast<long long>(kConvertThreads)) {
    const int row = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<long long>(row) * per_row) * 8;
    const long long at = row * m.ld + c;
    const T* const src = static_cast<const T*>(m.src) + at;
    [[maybe_unused]] const size_t extent = stored_extent(m.rows, m.cols, m.ld);
    float v[8];
    if (m.aligned && c + 8 <= m.cols && GEMM_IN_EXTENT(at + 7, extent, err, kSiteBoundsRows)) {
      Raw<T, 8> raw;
      raw.load_once(src);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = raw.at(j);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = c + j < m.cols && GEMM_IN_EXTENT(at + j, extent, err, kSiteBoundsRows) ? to_f32(src[j]) : 0.0f;
    }
    bf16* const out = m.dst + row * m.ld_dst + c;
    if constexpr (sizeof(T) == 2) {
      store_vec<bf16, 8>(out, v);
    } else {
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
    }
  }
}

// Both operands at once: the first `x_ctas` CTAs bring x back, the others
// prepare dy (rows 4096, 1024 x 1024 fp32: the whole call 41 us, 44 with two
// launches).
template <class T>
__global__ void __launch_bounds__(kConvertThreads) operands_kernel(const ConvertArgs x, const SplitArgs dy, unsigned x_ctas) {
  grid_launch_dependents();
  grid_dependency_wait();
  if (blockIdx.x < x_ctas)
    restore_rows<bf16, true>(x, blockIdx.x, x_ctas);
  else
    split_rows<T>(dy, blockIdx.x - x_ctas, gridDim.x - x_ctas, x.err);
}

// ---------------------------------------------------------------- host side
constexpr int kMost = INT_MAX - 1024;    // tiles and pieces rounded up stay within an int

size_t type_size(int type) { return type == GEMM_F32_TYPE_F32 ? 4 : 2; }

bool aligned_to(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool on_boundaries(const void* p, long long ld, size_t size) { return aligned_to(p, 16) && ld * size % 16 == 0; }

size_t matrix_bytes(long long rows, long long width, long long ld, size_t size) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * ld + width) * size : 0;
}

bool addressable(long long rows, long long ld) { return rows == 0 || ld <= LLONG_MAX / 8 / rows; }

bool type_ok(int type) { return type == GEMM_F32_TYPE_F32 || type == GEMM_F32_TYPE_BF16; }

bool matrix_ok(const void* p, long long ld, long long rows, int width, size_t size) {
  return p && aligned_to(p, size) && ld >= width && addressable(rows, ld);
}

bool saved_ok(const void* codes, long long ld_codes, const void* exponents, long long ld_exponents, long long rows,
              int width) {
  return codes && exponents && on_boundaries(codes, ld_codes, 1) && on_boundaries(exponents, ld_exponents, 1) &&
         ld_codes >= (width + 31LL) / 32 * 32 && ld_exponents >= (width + 31LL) / 32 && addressable(rows, ld_codes) &&
         addressable(rows, ld_exponents);
}

// A matrix apart from 8-bit rows.
bool apart(const void* p, size_t bytes, const void* codes, long long ld_codes, const void* exponents,
           long long ld_exponents, long long rows) {
  return !ranges_overlap(p, bytes, codes, static_cast<size_t>(rows) * ld_codes) &&
         !ranges_overlap(p, bytes, exponents, static_cast<size_t>(rows) * ld_exponents);
}

// Pieces of the rows, and as many CTAs as there is work for: a fixed number
// would leave the last ones of a wave alone.  `spare`: columns that rows which
// start above a boundary are taken to be longer by.
unsigned plan_convert(ConvertArgs& a, int flight, int spare) {
  a.pieces = static_cast<int>((a.width - 1LL + spare) / kPiece + 1);
  const long long per_cta = kConvertThreads / 32 * flight;
  const long long ctas = a.rows > LLONG_MAX / a.pieces ? LLONG_MAX : (a.rows * a.pieces - 1) / per_cta + 1;
  return static_cast<unsigned>(std::min<long long>(ctas, INT_MAX));
}

template <class Kernel, class... Args>
int launch(Kernel kernel, unsigned grid, cudaStream_t stream, int* launches, const Args&... args) {
  if (launch_dependent(kernel, dim3(grid), dim3(kConvertThreads), 0, stream, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  ++*launches;
  return GEMM_F32_OK;
}

struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" int gemm_f32_checkpoint(int type, long long rows, int width, const void* x, long long ldx,
                                   unsigned char* codes, long long ld_codes, unsigned char* exponents,
                                   long long ld_exponents, gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!type_ok(type) || rows < 0 || width < 1 || width > kMost) return GEMM_F32_EINVAL;
  if (rows == 0) return GEMM_F32_OK;
  const size_t es = type_size(type);
  if (!matrix_ok(x, ldx, rows, width, es) || !saved_ok(codes, ld_codes, exponents, ld_exponents, rows, width))
    return GEMM_F32_EINVAL;
  if (!apart(x, matrix_bytes(rows, width, ldx, es), codes, ld_codes, exponents, ld_exponents, rows) ||
      ranges_overlap(codes, static_cast<size_t>(rows) * ld_codes, exponents, static_cast<size_t>(rows) * ld_exponents))
    return GEMM_F32_EINVAL;
  int device = 0, num_sms = 0, launches = 0;
  ConvertArgs a = {rows, width, x, nullptr, ldx, codes, ld_codes, exponents, ld_exponents, 0, nullptr};
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  const bool vec = on_boundaries(x, ldx, es) && width * es % 16 == 0;
  const int flight = type == GEMM_F32_TYPE_BF16 && vec ? keep_flight<bf16, true>() : keep_flight<float, true>();
  const unsigned grid = plan_convert(a, flight, 0);
  const auto kernel = type == GEMM_F32_TYPE_F32 ? vec ? checkpoint_kernel<float, true> : checkpoint_kernel<float, false>
                                                : vec ? checkpoint_kernel<bf16, true> : checkpoint_kernel<bf16, false>;
  const int rc = launch(kernel, grid, reinterpret_cast<cudaStream_t>(stream_handle), &launches, a);
  if (rc == GEMM_F32_OK) note_launches(launches, "checkpoint_kernel");
  return rc;
}

extern "C" int gemm_f32_restore(int type, long long rows, int width, const unsigned char* codes, long long ld_codes,
                                const unsigned char* exponents, long long ld_exponents, void* out, long long ldo,
                                gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!type_ok(type) || rows < 0 || width < 1 || width > kMost) return GEMM_F32_EINVAL;
  if (rows == 0) return GEMM_F32_OK;
  const size_t es = type_size(type);
  if (!matrix_ok(out, ldo, rows, width, es) || !saved_ok(codes, ld_codes, exponents, ld_exponents, rows, width) ||
      !apart(out, matrix_bytes(rows, width, ldo, es), codes, ld_codes, exponents, ld_exponents, rows))
    return GEMM_F32_EINVAL;
  int device = 0, num_sms = 0, launches = 0;
  ConvertArgs a = {rows,     width, nullptr, out, ldo, const_cast<uint8_t*>(codes), ld_codes, const_cast<uint8_t*>(exponents),
                   ld_exponents, 0,     nullptr};
  if (!current_device(&device, &num_sms, &a.err)) return GEMM_F32_EDEVICE;
  const bool vec = on_boundaries(out, ldo, es) && width * es % 16 == 0;
  const unsigned grid = plan_convert(a, kRestoreFlight, vec ? 0 : 7);
  const auto kernel = type == GEMM_F32_TYPE_F32 ? vec ? restore_kernel<float, true> : restore_kernel<float, false>
                                                : vec ? restore_kernel<bf16, true> : restore_kernel<bf16, false>;
  const int rc = launch(kernel, grid, reinterpret_cast<cudaStream_t>(stream_handle), &launches, a);
  if (rc == GEMM_F32_OK) note_launches(launches, "restore_kernel");
  return rc;
}

namespace gemm_f32_impl {
namespace {

struct WeightGrad {
  bool f32;                              // dy
  int rows, width, out;
  const void* dy;
  long long lddy;
  const uint8_t* codes;
  long long ld_codes;
  const uint8_t* exponents;
  long long ld_exponents;
  bool dw_f32;
  void* dw;
  long long lddw;
  bool accumulate;
};

int run_weight_grad(const WeightGrad& c, cudaStream_t stream, int* launches) {
  int device = 0, num_sms = 0;
  unsigned* err = nullptr;
  if (!current_device(&device, &num_sms, &err)) return GEMM_F32_EDEVICE;
  const int parts = c.f32 ? 3 : 1;
  const long long ldx = (c.width + 7LL) / 8 * 8;
  const bool packed = c.f32 || !on_boundaries(c.dy, c.lddy, 2);
  const long long lddy = packed ? (c.out + 7LL) / 8 * 8 : c.lddy;
  Layout layout;
  const size_t at_x = layout.take(static_cast<size_t>(c.rows) * ldx * 2);
  const size_t at_dy = packed ? layout.take(static_cast<size_t>(c.rows) * lddy * 2 * parts) : 0;
  const size_t at_partials = layout.take(half_gemm_scratch(c.out, c.width, c.rows, parts, num_sms, !c.f32));
  char* const scratch = static_cast<char*>(acquire_scratch(device, stream, layout.bytes));
  if (!scratch) return GEMM_F32_ESCRATCH;
  ConvertArgs x = {c.rows,      static_cast<int>(ldx), nullptr, scratch + at_x, ldx, const_cast<uint8_t*>(c.codes), c.ld_codes,
                   const_cast<uint8_t*>(c.exponents), c.ld_exponents,   0,       err};
  const unsigned x_ctas = plan_convert(x, kRestoreFlight, 0);
  const long long plane = lddy * c.rows;
  int rc;
  if (packed) {
    const SplitArgs dy = {c.dy, reinterpret_cast<bf16*>(scratch + at_dy), c.lddy, lddy, plane, plane / 8, c.rows, c.out,
                          on_boundaries(c.dy, c.lddy, c.f32 ? 4 : 2)};
    const long long all = (dy.vectors - 1) / kConvertThreads + 1;
    const unsigned dy_ctas = static_cast<unsigned>(std::min<long long>(all, 16LL * num_sms));
    const unsigned first = std::min(x_ctas, 1u << 30);   // the sum stays within a grid
    rc = c.f32 ? launch(operands_kernel<float>, first + dy_ctas, stream, launches, x, dy, first)
               : launch(operands_kernel<bf16>, first + dy_ctas, stream, launches, x, dy, first);
  } else {
    rc = launch(restore_kernel<bf16, true>, x_ctas, stream, launches, x);
  }
  if (rc != GEMM_F32_OK) return rc;
  HalfGemm g = {};
  g.M = c.out;
  g.N = c.width;
  g.K = c.rows;
  g.parts = parts;
  g.a = {packed ? scratch + at_dy : c.dy, lddy, plane, true};
  g.b = {scratch + at_x, ldx, 0, true};
  g.b_whole = true;
  g.summed = !c.f32;
  g.c = c.dw;
  g.ldc = c.lddw;
  g.c_f32 = c.dw_f32;
  if (c.accumulate) {
    g.add = static_cast<const float*>(c.dw);
    g.ldadd = c.lddw;
  }
  g.partials = reinterpret_cast<float*>(scratch + at_partials);
  g.num_sms = num_sms;
  g.device = device;
  g.err = err;
  return launch_half_gemm(g, stream, launches);
}

}  // namespace
}  // namespace gemm_f32_impl

extern "C" int gemm_f32_weight_grad(int type, long long rows, int width, int out, const void* dy, long long lddy,
                                    const unsigned char* codes, long long ld_codes, const unsigned char* exponents,
                                    long long ld_exponents, int dw_type, void* dw, long long lddw, int accumulate,
                                    gemm_f32_stream_t stream_handle) {
  note_launches(0, "none");
  if (!type_ok(type) || (dw_type != type && dw_type != GEMM_F32_TYPE_F32)) return GEMM_F32_EINVAL;
  if (accumulate != 0 && (accumulate != 1 || dw_type != GEMM_F32_TYPE_F32)) return GEMM_F32_EINVAL;
  if (rows < 0 || rows > kMost || width < 1 || width > kMost || out < 1 || out > kMost) return GEMM_F32_EINVAL;
  const size_t es = type_size(type), ds = type_size(dw_type);
  if (!matrix_ok(dw, lddw, out, width, ds)) return GEMM_F32_EINVAL;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
  int launches = 0;
  if (rows == 0) {
    int device = 0, num_sms = 0;
    unsigned* err = nullptr;
    if (accumulate) return GEMM_F32_OK;
    if (!current_device(&device, &num_sms, &err)) return GEMM_F32_EDEVICE;
    if (cudaMemset2DAsync(dw, lddw * ds, 0, width * ds, out, stream) != cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    note_launches(1, "memset");
    return GEMM_F32_OK;
  }
  const size_t dw_bytes = matrix_bytes(out, width, lddw, ds);
  if (!matrix_ok(dy, lddy, rows, out, es) || !saved_ok(codes, ld_codes, exponents, ld_exponents, rows, width) ||
      !apart(dw, dw_bytes, codes, ld_codes, exponents, ld_exponents, rows) ||
      ranges_overlap(dw, dw_bytes, dy, matrix_bytes(rows, out, lddy, es)))
    return GEMM_F32_EINVAL;
  const WorkspaceCall call;
  const WeightGrad c = {type == GEMM_F32_TYPE_F32, static_cast<int>(rows), width, out, dy, lddy, codes, ld_codes,
                        exponents, ld_exponents, dw_type == GEMM_F32_TYPE_F32, dw, lddw, accumulate != 0};
  const int rc = run_weight_grad(c, stream, &launches);
  if (rc == GEMM_F32_OK) note_launches(launches, "half_gemm_kernel");
  return rc;
}
