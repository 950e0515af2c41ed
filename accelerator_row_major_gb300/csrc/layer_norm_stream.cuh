// Layer norm over many rows: the streaming kernels (sm_103a).
//
// Each group of G threads works on one row at a time and keeps the next rows
// in a ring in shared memory, filled by bulk copies (cp.async.bulk on
// mbarriers).  One CTA of 512 threads (or the groups that 512 make) per SM.
// Threads hold up to 32 elements of a row in the forward pass and 16 in the
// gradient: what a row costs besides its elements (reductions, barriers) is then
// paid by few warps, and the arithmetic is done two elements at a time
// (f32x2).  With 8 elements a thread the issue of instructions bound both
// kernels (65536 x 1024 bfloat16: 60 and 91 us against 47 and 70; the copy
// rate allows 40 and 59).  What the row leaves of a group's elements costs as
// much as the row's, so besides the powers of 2 there are groups that hold
// 3/4 of them: 24 elements a thread, or in the gradient, whose registers hold
// no more than 16, three warps for four (1280 columns of 52428 rows in
// bfloat16: 52 and 79 us against 59 and 100 with room for 2048).
//
// RAGGED: rows that do not all start and end on 16-byte boundaries.  A row is
// copied from the boundary below its start to the one above its end (never
// beyond the matrix: what is left at its first and last bytes, in the first
// and the last row or in rows closer than 16 bytes, is copied by a thread), and threads take the 16-byte vectors of that copy, of which the
// first and the last hold elements of other rows.  Rows start 0 to 14 bytes
// above a boundary, each of 16 / gcd(16, stride) rows differently; the number
// of groups is a multiple of that, so that a group meets rows of one start
// only, and its threads keep their columns.  (65536 x 777 fp32: 71 and 103 us,
// copies 60 and 90; 65536 x 1001 bfloat16: 65 and 90 us, copies 39 and 58,
// bound by the instructions that the rows' ends cost.)
//
// CTAS > 1 (gradient of rows wider than 8192): a cluster shares a row, each
// CTA a slice of its columns (cut on 16-byte boundaries), and exchanges the two sums of the row through
// distributed shared memory: asynchronous stores that a barrier at their
// destination counts.  A barrier of the cluster in their place would wait for
// every store of dx in flight (4096 x 16384 bfloat16 133 us against 90, fp32
// 173 against 139).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "pair_common.cuh"
#include "row_common.cuh"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

using bf16 = __nv_bfloat16;

struct NormArgs {
  long long rows;
  int width;
  const void* x;
  const void* dy;          // gradient only
  long long ldx, lddy;
  const void* weight;
  const void* bias;        // forward only
  float eps;
  void* out;               // y, or dx
  long long ldo;
  float* mean;             // written by the forward pass, read by the gradient
  float* rstd;
  float* partials;         // gradient: [CTA][2][width]
  float* row_sums;         // gradient of wide rows: [rows][2]
  unsigned* err;
};

template <class T>
__device__ __forceinline__ bool row_ok(const NormArgs& a, size_t at, int n, long long ld) {
  return GEMM_IN_EXTENT(at + n - 1, stored_extent(a.rows, a.width, ld), a.err, kSiteBoundsRows);
}

// ---------------------------------------------------------------- rings
constexpr int stream_threads(int g) { return 512 / g * g; }   // whole groups
constexpr size_t kStreamBytes = 200 * 1024;
constexpr int kMostStages = 8;

// Shared memory of one row of a ring.
__host__ __device__ __forceinline__ size_t ring_row_bytes(int width, size_t size, bool ragged) {
  return ragged ? (width * size + 15) / 16 * 16 + 16 : width * size;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// The ring of one group: ARRAYS rows per stage (x, or x and dy), filled for
// the group's rows first, first + step, ..., `stages` ahead.  Of each row the
// `width` elements from column `col0` on: all of it, or where `ctas` CTAs
// share a row the slice of CTA `rank`.  Slices are cut on 16-byte boundaries,
// so that no CTA has more than `slice` elements of whole blocks to hold: a row
// that starts above a boundary leaves the first CTA so many elements fewer.
template <class T, int ARRAYS, bool RAGGED>
struct RowRing {
  const NormArgs& a;
  uint8_t* data;
  uint32_t bars, row_bytes;
  uint32_t around = 0;          // RAGGED: bytes of the 16-byte blocks around a row of this group
  int width, col0, stages, s = 0;
  uint32_t ph = 0;
  bool lost = false;
  long long next, step;

  __device__ __forceinline__ RowRing(const NormArgs& args, uint8_t* smem, int group, int groups, int st,
                                     int slice, int rank, int ctas)
      : a(args), width(min(slice, args.width)), col0(0), stages(st) {   // a value of its own, not a parameter: fewer spills
    row_bytes = static_cast<uint32_t>(ring_row_bytes(slice, sizeof(T), RAGGED));
    data = smem + static_cast<size_t>(group) * st * ARRAYS * row_bytes;
    bars = smem_addr(smem) + static_cast<uint32_t>(groups) * st * ARRAYS * row_bytes +
           static_cast<uint32_t>(group) * st * 8u;
    step = static_cast<long long>(gridDim.x / ctas) * groups;
    next = static_cast<long long>(blockIdx.x / ctas) * groups + group;
    if (ctas > 1) {
      const int lead = shift();            // of the whole row
      if (rank > 0) col0 = rank * slice - lead;
      width = min(rank > 0 ? slice : slice - lead, args.width - col0);
    }
    if (RAGGED) around = ((shift() + width) * static_cast<uint32_t>(sizeof(T)) + 15u) & ~15u;
  }
  // One thread of the group, before the group's first barrier.
  __device__ __forceinline__ void init() {
    for (int i = 0; i < stages; ++i) mbar_init(bars + 8u * i, 1);
    fence_mbar_init();
  }
  __device__ __forceinline__ const T* source(int array, long long row) const {
    return (array == 0 ? static_cast<const T*>(a.x) + row * a.ldx
                       : static_cast<const T*>(a.dy) + row * a.lddy) + col0;
  }
  // One thread: the copies of row `next` into stage `at`.
  __device__ __forceinline__ void load(int at) {
    if (next < a.rows) {
      const uint32_t bar = bars + 8u * at;
      uint8_t* const dst = data + static_cast<size_t>(at) * ARRAYS * row_bytes;
      if (RAGGED && inner()) {                 // the blocks around the row are the matrix's
        mbar_arrive_expect_tx(bar, ARRAYS * around);
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
          bulk_load(smem_addr(dst) + i * row_bytes,
                    reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(source(i, next)) & ~uintptr_t{15}),
                    around, bar);
      } else if constexpr (RAGGED) {
        uint32_t bytes[ARRAYS];
        uintptr_t from[ARRAYS];
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i) edges(i, dst + i * row_bytes, from[i], bytes[i]);
        mbar_arrive_expect_tx(bar, ARRAYS == 2 ? bytes[0] + bytes[ARRAYS - 1] : bytes[0]);
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
          if (bytes[i])
            bulk_load(smem_addr(dst) + i * row_bytes +
                          static_cast<uint32_t>(from[i] - (reinterpret_cast<uintptr_t>(source(i, next)) & ~uintptr_t{15})),
                      reinterpret_cast<const void*>(from[i]), bytes[i], bar);
      } else {
        const uint32_t bytes = static_cast<uint32_t>(width * sizeof(T));
        mbar_arrive_expect_tx(bar, ARRAYS * bytes);
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
          bulk_load(smem_addr(dst) + i * row_bytes, source(i, next), bytes, bar);
      }
    }
    next += step;
  }
  // Whether row `next` has a whole block of the matrix before it and one behind
  // it: not the first row nor the last, nor rows that lie closer than a block.
  __device__ __forceinline__ bool inner() const {
    constexpr long long kBlock = 16 / static_cast<int>(sizeof(T));
    if (next == 0 || next == a.rows - 1 || a.ldx < kBlock || (ARRAYS == 2 && a.lddy < kBlock)) return false;
#ifdef GEMM_BOUNDS_CHECK
    for (int i = 0; i < ARRAYS; ++i) {
      const long long ld = i == 0 ? a.ldx : a.lddy;
      const uintptr_t lowest = reinterpret_cast<uintptr_t>(i == 0 ? a.x : a.dy);
      const uintptr_t from = reinterpret_cast<uintptr_t>(source(i, next)) & ~uintptr_t{15};
      // what lies before the matrix wraps round to beyond it
      const size_t bytes = stored_extent(a.rows, a.width, ld) * sizeof(T);
      if (!GEMM_IN_EXTENT(from - lowest, bytes, a.err, kSiteBoundsRows) ||
          !GEMM_IN_EXTENT(from + around - 1 - lowest, bytes, a.err, kSiteBoundsRows))
        return false;
    }
#endif
    return true;
  }
  // The 16-byte blocks of row `next` that lie within the matrix go by one bulk
  // copy (`bytes` from `from` on); its elements outside them, near the matrix's
  // two ends only, are copied here.
  __device__ __forceinline__ void edges(int array, uint8_t* dst, uintptr_t& from, uint32_t& bytes) {
    const T* const row = source(array, next);
    const uintptr_t first = reinterpret_cast<uintptr_t>(row), last = first + width * sizeof(T);
    const long long ld = array == 0 ? a.ldx : a.lddy;
    const uintptr_t lowest = reinterpret_cast<uintptr_t>(array == 0 ? a.x : a.dy);
    const uintptr_t end = lowest + stored_extent(a.rows, a.width, ld) * sizeof(T);
    uintptr_t lo = first & ~uintptr_t{15}, hi = (last + 15) & ~uintptr_t{15};
    if (lo < lowest) lo += 16;
    if (hi > end) hi -= 16;
    T* const at = reinterpret_cast<T*>(dst + (first & 15));
    if (lo >= hi) {       // no whole block
      lo = hi = first;
      for (int d = 0; d < width; ++d) at[d] = row[d];
    } else {
      for (uintptr_t p = first; p < lo; p += sizeof(T)) at[(p - first) / sizeof(T)] = *reinterpret_cast<const T*>(p);
      for (uintptr_t p = hi; p < last; p += sizeof(T)) at[(p - first) / sizeof(T)] = *reinterpret_cast<const T*>(p);
    }
    from = lo;
    bytes = static_cast<uint32_t>(hi - lo);
  }
  // A wait that runs out is recorded, and the thread goes on (the result is
  // undefined, as the status says): the group's barriers need all of it.  The
  // one that issues the copies issues no more.
  __device__ __forceinline__ void wait() {
    if (!lost) lost = !mbar_wait(bars + 8u * s, ph, a.err, kSiteTransformFull);
  }
  // The issuing thread, after its last row (`row` is beyond it): where it gave
  // up, it waits, again with a limit, for its copies still in flight, which
  // would land in memory that is no longer the kernel's.  They are those of the
  // rows from next - stages step on; the stage and phase of the first follow
  // from those of `row`.
  __device__ __forceinline__ void finish(long long row) const {
    if (!lost) return;
    const long long first = next - stages * step, since = (row - first) / step;
    int at = static_cast<int>(((s - since) % stages + stages) % stages);
    uint32_t parity = ph ^ (static_cast<uint32_t>((at + since) / stages) & 1u);
    for (int k = 0; k < stages && first + k * step < a.rows; ++k) {
      mbar_wait(bars + 8u * at, parity, a.err, kSiteDrainTma);
      if (++at == stages) {
        at = 0;
        parity ^= 1u;
      }
    }
  }
  // The stage's copy of an array's row.
  __device__ __forceinline__ const uint8_t* at(int array) const {
    return data + (static_cast<size_t>(s) * ARRAYS + array) * row_bytes;
  }
  // Elements by which the group's rows (or slices) start above a 16-byte boundary.
  __device__ __forceinline__ int shift() const {
    return RAGGED ? static_cast<int>((reinterpret_cast<uintptr_t>(source(0, next)) & 15) / sizeof(T)) : 0;
  }
  __device__ __forceinline__ void advance() {
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// ---------------------------------------------------------------- a thread's part of a row
// RAGGED: which elements of a 16-byte vector are the row's, as bits and as
// factors.  Entry 0: all; entry e < 8: all but the first e; entry 8 + n: the
// first n.
template <class T>
struct Edges {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  T cut[16][2][kVec];                    // of each warp: its cut vectors, as stored
  uint4 bits[16];
  float ones[16][kVec];

  __device__ __forceinline__ void fill() {
    const int e = threadIdx.x;
    if (e >= 16) return;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const bool in = e < 8 ? i >= e : i < e - 8;
      ones[e][i] = in ? 1.0f : 0.0f;
      if (in) w[i * static_cast<int>(sizeof(T)) / 4] |= sizeof(T) == 4 ? ~0u : 0xFFFFu << (16 * (i & 1));
    }
    bits[e] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ void keep(uint4& q, const uint4& bits) {
  q.x &= bits.x;
  q.y &= bits.y;
  q.z &= bits.z;
  q.w &= bits.w;
}

// NP pairs of elements: vector i of thread t holds the elements from column
// (i G + t) VEC - shift on.  Of a ragged row the first vector of thread 0 and
// vector i_last of one thread are cut.  All threads take these two vectors
// through masks (of all elements, but for the threads that hold the cut ones):
// less work for a warp than branches of one thread (65536 x 1001 bfloat16:
// 77 and 108 us against 75 and 113, then 69 and 87 with the rows inside the
// matrix copied without a look at its ends, 62 forward with staged stores).
template <class T, int G, int NP, bool RAGGED, bool STAGED>
struct Part {
  static constexpr int kPer = 8 / static_cast<int>(sizeof(T));   // pairs per vector
  static constexpr int kVec = 2 * kPer;
  static constexpr int NV = NP / kPer;
  Edges<T>& edges;
  int width, first;                      // columns of the row, column of vector 0
  int i_last = -1;
  int head = 0, tail = 0;                // entries of the masks
  int cut_col = -1;                      // STAGED: column of the element of a cut vector that this lane stores

  __device__ __forceinline__ Part(Edges<T>& e, int w, int shift, int t)
      : edges(e), width(w), first(t * kVec - shift) {
    if constexpr (RAGGED) {
      const int last = (w + shift - 1) / kVec, part = (w + shift) % kVec;
      i_last = last / G;
      if (t == 0) head = shift;
      if (t == last % G && part != 0) tail = 8 + part;
      if constexpr (STAGED) {           // lanes 0 .. VEC - 1 the first vector, the next VEC the last
        const int at = t % kVec, of = t % 32 / kVec;
        const bool both = last == 0 && part != 0;              // one vector, cut at both ends
        if (of == 0 && t < 32 && at >= shift && shift != 0 && !both) cut_col = at - shift;
        if (of == 1 && t / 32 == last % G / 32 && at < part && (last != 0 || at >= shift))
          cut_col = last * kVec + at - shift;
      }
    }
  }
  __device__ __forceinline__ int col(int i) const { return i * (G * kVec) + first; }
  __device__ __forceinline__ bool any(int i) const {
    return RAGGED ? col(i) + kVec > 0 && col(i) < width : col(i) < width;
  }
  __device__ __forceinline__ bool in(int d) const { return d >= 0 && d < width; }

  // The row's elements, 0 for what lies outside it.
  __device__ __forceinline__ void load(const uint8_t* copy, int t, Pair (&x)[NP]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pair v[kPer];
      if constexpr (RAGGED) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (any(i)) q = *reinterpret_cast<const uint4*>(copy + (i * G + t) * 16);
        if (i == 0) keep(q, edges.bits[head]);
        if (i == i_last) keep(q, edges.bits[tail]);
        pairs_of<T>(q, v);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = 0;
        if (any(i)) pairs_of<T>(*reinterpret_cast<const uint4*>(copy + (i * G + t) * 16), v);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[i * kPer + j] = v[j];
    }
  }

  // sum plus the squares of a ragged row's elements; what lies outside is finite.
  __device__ __forceinline__ Pair add_squares(const Pair (&x)[NP], Pair sum) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pair v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = x[i * kPer + j];
      if (i == 0) scale(v, edges.ones[head]);
      if (i == i_last) scale(v, edges.ones[tail]);
      if (any(i)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum = fma2(v[j], x[i * kPer + j], sum);
      }
    }
    return sum;
  }
  static __device__ __forceinline__ void scale(Pair (&v)[kPer], const float* by) {
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
      const float4 f = *reinterpret_cast<const float4*>(by + 2 * j);
      v[j] = mul2(v[j], pair_of(f.x, f.y));
      v[j + 1] = mul2(v[j + 1], pair_of(f.z, f.w));
    }
  }

  template <class WT>
  __device__ __forceinline__ void load_weights(const void* p, float none, Pair (&w)[NP]) const {
    const WT* const v = static_cast<const WT*>(p);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) f[j] = none;
      if constexpr (RAGGED) {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (p && in(col(i) + j)) f[j] = to_f32(v[col(i) + j]);
      } else {
        if (p && any(i)) load_cached<WT, kVec>(v + col(i), f);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) w[i * kPer + j] = pair_of(f[2 * j], f[2 * j + 1]);
    }
  }

  // Cut vectors: staged, through shared memory, from where as many lanes
  // store an element each; else a few stores by the thread that holds them,
  // which take a warp more instructions but no register (65472 x 1025
  // bfloat16 forward 81 us against 97; gradient of 32880 x 2041 97 against 87).
  __device__ __forceinline__ void store(T* y, const Pair (&x)[NP]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pair v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = x[i * kPer + j];
      bool whole = any(i);
      if constexpr (RAGGED) {
        const bool from = i == 0 && head != 0, to = i == i_last && tail != 0;
        if constexpr (STAGED) {
          if (from) store_pairs(edges.cut[threadIdx.x / 32][0], v);
          if (to) store_pairs(edges.cut[threadIdx.x / 32][1], v);
          if (from || to) whole = false;
        } else if (from || to) {
          store_cut(y + col(i), v, from ? head : 0, to ? tail - 8 : kVec);
          whole = false;
        }
      }
      if (whole) store_pairs(y + col(i), v);
    }
    if constexpr (STAGED) {
      __syncwarp();
      if (cut_col >= 0) y[cut_col] = (&edges.cut[threadIdx.x / 32][0][0])[threadIdx.x % 32];
      __syncwarp();                     // read, before the next row's are written
    }
  }
  // Elements [b, e) of the vector at y, one of whose ends is the vector's (of
  // a row of a few elements neither may be), as 2, 4 and 8 bytes.
  static __device__ __forceinline__ void store_cut(T* y, const Pair (&v)[kPer], int b, int e) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      float f, g;
      unpair(v[j], f, g);
      if constexpr (sizeof(T) == 4) {
        w[2 * j] = __float_as_uint(f);
        w[2 * j + 1] = __float_as_uint(g);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f, g);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    const auto put = [&](int j) {                               // element j
      if constexpr (sizeof(T) == 4)
        reinterpret_cast<uint32_t*>(y)[j] = w[j];
      else
        reinterpret_cast<uint16_t*>(y)[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    };
    if (b != 0 && e != kVec) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j >= b && j < e) put(j);
      return;
    }
    constexpr int kWord = 4 / static_cast<int>(sizeof(T));      // elements in 4 bytes
    uint32_t* const words = reinterpret_cast<uint32_t*>(y);
    // the odd element, the odd word and the half that make up the part
    const int n = e - b, odd_at = b != 0 ? b : e - 1;
    const int word = b != 0 ? (b + kWord - 1) / kWord : e / kWord - 1;   // of the part's whole words, the outermost
    const int whole = n / kWord;                                         // whole words: 0 .. 3
    if (kWord == 2 && (n & 1)) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j == odd_at) put(j);
    }
    if (whole & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == word) words[j] = w[j];
    }
    if (whole & 2) {
      if (b != 0)
        reinterpret_cast<uint2*>(y)[1] = make_uint2(w[2], w[3]);
      else
        reinterpret_cast<uint2*>(y)[0] = make_uint2(w[0], w[1]);
    }
  }
};

// ---------------------------------------------------------------- kernels
template <class T, class WT, int G, int NP, bool RAGGED>
__global__ void __launch_bounds__(stream_threads(G), 1)
    layer_norm_stream_kernel(NormArgs a, int stages, int slice) {
  constexpr int kGroups = stream_threads(G) / G;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ Edges<T> edges;
  __shared__ float part[2][kGroups][G / 32];
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  RowRing<T, 1, RAGGED> ring(a, smem_rows, group, kGroups, stages, slice, 0, 1);
  if (t == 0) ring.init();
  if (RAGGED) edges.fill();
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  const Part<T, G, NP, RAGGED, RAGGED> mine(edges, a.width, ring.shift(), t);
  long long row = ring.next;
  if (t == 0)
    for (int i = 0; i < stages; ++i) ring.load(i);
  const float inv = 1.0f / static_cast<float>(a.width);
  Pair w[NP], b[NP];
  mine.template load_weights<WT>(a.weight, 1.0f, w);
  mine.template load_weights<WT>(a.bias, 0.0f, b);
  for (; row < a.rows; row += ring.step) {
    ring.wait();
    Pair x[NP], sum = 0;
    mine.load(ring.at(0), t, x);
#pragma unroll
    for (int q = 0; q < NP; ++q) sum = add2(sum, x[q]);
    float s[1] = {sum_of(sum)};
    group_sum<1, G>(s, part[0][group], group);
    if (t == 0 && !ring.lost) ring.load(ring.s);   // the group has read this stage
    ring.advance();
    const float mean = s[0] * inv;
    const Pair minus = pair_of(-mean, -mean);
#pragma unroll
    for (int q = 0; q < NP; ++q) x[q] = add2(x[q], minus);
    sum = 0;
    if constexpr (RAGGED) {
      sum = mine.add_squares(x, sum);
    } else {
#pragma unroll
      for (int q = 0; q < NP; ++q)
        if (mine.any(q / mine.kPer)) sum = fma2(x[q], x[q], sum);
    }
    s[0] = sum_of(sum);
    group_sum<1, G>(s, part[1][group], group);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    const Pair by = pair_of(rstd, rstd);
#pragma unroll
    for (int q = 0; q < NP; ++q) x[q] = fma2(mul2(x[q], by), w[q], b[q]);
    if (GEMM_IN_EXTENT(row * a.ldo + a.width - 1, stored_extent(a.rows, a.width, a.ldo), a.err, kSiteBoundsRows))
      mine.store(static_cast<T*>(a.out) + row * a.ldo, x);
  }
  if (t == 0) ring.finish(row);
}

// Two floats into the shared memory of another CTA of the cluster, counted by
// a barrier there.
__device__ __forceinline__ void store_async(uint32_t to, float x, float y, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
               "f"(x), "f"(y), "r"(bar)
               : "memory");
}

template <class T, class WT, int G, int NP, bool RAGGED, int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(stream_threads(G), 1)
    layer_norm_grad_stream_kernel(NormArgs a, int stages, int slice) {
  constexpr int kThreads = stream_threads(G);
  constexpr int kGroups = kThreads / G;
  static_assert(CTAS == 1 || kGroups == 1, "a cluster works on one row");
  extern __shared__ __align__(128) uint8_t smem_rows[];
  __shared__ Edges<T> edges;
  __shared__ float part[2][kGroups][2 * (G / 32)];
  __shared__ float2 shared_sums[2][CTAS];              // of the CTAs of the cluster
  __shared__ uint64_t shared_bars[2];
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_rank()) : 0;
  RowRing<T, 2, RAGGED> ring(a, smem_rows, group, kGroups, stages, slice, rank, CTAS);
  const int width = ring.width, col0 = ring.col0;      // of this CTA's slice
  const uint32_t bars = smem_addr(shared_bars);
  if (threadIdx.x == 0 && CTAS > 1)
    for (int i = 0; i < 2; ++i) mbar_init(bars + 8u * i, 1);
  if (t == 0) ring.init();
  if (RAGGED) edges.fill();
  __syncthreads();
  if (CTAS > 1) cluster_sync();              // every CTA of the cluster runs
  grid_launch_dependents();
  grid_dependency_wait();
  const Part<T, G, NP, RAGGED, false> mine(edges, width, ring.shift(), t);
  long long row = ring.next;
  if (t == 0)
    for (int i = 0; i < stages; ++i) ring.load(i);
  const float inv = 1.0f / static_cast<float>(a.width);
  Pair w[NP], dw[NP], db[NP];
  mine.template load_weights<WT>(a.weight ? static_cast<const WT*>(a.weight) + col0 : nullptr, 1.0f, w);
#pragma unroll
  for (int q = 0; q < NP; ++q) dw[q] = db[q] = 0;
  uint32_t flip = 0, round = 0;
  float mean = 0.0f, rstd = 0.0f;
  if (row < a.rows) {
    mean = __ldg(a.mean + row);
    rstd = __ldg(a.rstd + row);
  }
  for (; row < a.rows; row += ring.step) {
    ring.wait();
    float mean_n = 0.0f, rstd_n = 0.0f;      // the next row's, under this row's work
    if (row + ring.step < a.rows) {
      mean_n = __ldg(a.mean + row + ring.step);
      rstd_n = __ldg(a.rstd + row + ring.step);
    }
    const Pair minus = pair_of(-mean, -mean), by = pair_of(rstd, rstd);
    // c = x - mean in place of hat = c rstd.  Outside the row dy is 0 and c
    // -mean: 0 in every sum, where hat might be infinite (times 0: not a
    // number).  Where rstd is 0, squares that overflowed, so are the hats.
    Pair c[NP], g[NP], sg = 0, sgc = 0;
    mine.load(ring.at(0), t, c);
    mine.load(ring.at(1), t, g);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      c[q] = add2(c[q], minus);
      dw[q] = fma2(mul2(g[q], by), c[q], dw[q]);
      db[q] = add2(db[q], g[q]);
      g[q] = mul2(g[q], w[q]);
      sg = add2(sg, g[q]);
      sgc = fma2(g[q], c[q], sgc);
    }
    float s[2] = {sum_of(sg), rstd != 0.0f ? sum_of(sgc) * rstd : 0.0f};
    group_sum<2, G>(s, part[flip][group], group);
    if (t == 0 && !ring.lost) ring.load(ring.s);   // the group has read this stage
    ring.advance();
    if constexpr (CTAS > 1) {                // every CTA adds the slices' sums in order
      if (t == 0) mbar_arrive_expect_tx(bars + 8u * flip, CTAS * 8u);
      if (t < CTAS)
        store_async(map_rank(smem_addr(&shared_sums[flip][rank]), static_cast<uint32_t>(t)), s[0], s[1],
                    map_rank(bars + 8u * flip, static_cast<uint32_t>(t)));
      if (!ring.lost) ring.lost = !mbar_wait_cluster(bars + 8u * flip, round, a.err, kSiteTransformFull);
      round ^= flip;                         // both have been waited for
      s[0] = s[1] = 0.0f;
#pragma unroll
      for (int i = 0; i < CTAS; ++i) {
        s[0] += shared_sums[flip][i].x;
        s[1] += shared_sums[flip][i].y;
      }
    }
    flip ^= 1;
    if (a.out) {
      const float c1 = -s[0] * inv, c2 = -s[1] * inv * rstd;
      const Pair minus_c1 = pair_of(c1, c1), minus_c2 = pair_of(c2, c2);
#pragma unroll
      for (int q = 0; q < NP; ++q) g[q] = mul2(fma2(c[q], minus_c2, add2(g[q], minus_c1)), by);
      if (GEMM_IN_EXTENT(row * a.ldo + a.width - 1, stored_extent(a.rows, a.width, a.ldo), a.err,
                         kSiteBoundsRows))
        mine.store(static_cast<T*>(a.out) + row * a.ldo + col0, g);
    }
    mean = mean_n;
    rstd = rstd_n;
  }
  if (t == 0) ring.finish(row);
  if (CTAS > 1) cluster_sync();              // no CTA leaves while another may write to it
  if (!a.partials) return;
  // the groups' column sums, added in group order: one row of partials per
  // CTA (or cluster); the rings make room
  float* const cols = reinterpret_cast<float*>(smem_rows);
  float* const to = a.partials + static_cast<size_t>(blockIdx.x / CTAS) * 2 * a.width + col0;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    float* const own = cols + group * width;
#pragma unroll
    for (int i = 0; i < mine.NV; ++i)
#pragma unroll
      for (int j = 0; j < mine.kPer; ++j) {
        const int q = i * mine.kPer + j, d = mine.col(i) + 2 * j;
        float u, v;
        unpair(which ? db[q] : dw[q], u, v);
        if (mine.in(d)) own[d] = u;
        if (mine.in(d + 1)) own[d + 1] = v;
      }
    __syncthreads();
    for (int d = threadIdx.x; d < width; d += kThreads) {
      float v = cols[d];
#pragma unroll
      for (int g2 = 1; g2 < kGroups; ++g2) v += cols[g2 * width + d];
      to[static_cast<size_t>(which) * a.width + d] = v;
    }
  }
}

}  // namespace
}  // namespace gemm_f32_impl
