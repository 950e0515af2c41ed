// Rows of several matrices at once, for the norms at a block's ends: a ring
// of rows in shared memory that bulk copies fill, a thread's part of a row,
// and sums over the threads that share one.
//
// A group of `lanes` threads (whole warps, as many as a row's columns need at
// NE elements a thread) works on one row at a time, or on two; a CTA has
// several groups where rows are narrow, and a cluster of CTAs shares a row,
// each a slice of its columns, where they are wide.  Lanes, groups, ring depth
// and cluster are the launch's: a width costs the next whole warp, not the next
// power of 2.
//
// The groups work on consecutive rows.  A stage of the ring holds a chunk of
// them: a row where rows are long, so that no group waits for another, several
// where they are short, so that the copies keep up.  Warps of their own issue
// the copies, a lane for each matrix (or for each matrix and row, where rows
// do not lie one behind the other): as work of the threads that compute, the
// copies' addresses were most of a row's time (65536 x 1024 bfloat16 forward
// 265 us against 157 with that alone changed, gradient 509 against 370).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block_norm.h"
#include "device_common.cuh"
#include "pair_common.cuh"
#include "row_common.cuh"
#include "saved_rows.cuh"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

using bf16 = __nv_bfloat16;

// ---------------------------------------------------------------- ring
// The first byte of a row's (or slice's) part of a matrix.
__device__ __forceinline__ uintptr_t first_byte(const RowSource& m, long long row, int col0) {
  return reinterpret_cast<uintptr_t>(m.p) + row * m.ld + (m.size ? col0 * m.size : col0 / kSavedBlock);
}

// What producer and consumers of a CTA's ring know alike.
struct RingPlace {
  uint8_t* data;
  uint32_t full, empty;                  // barriers: the copies have landed; all warps have read
  int col0, width;                       // of this CTA's slice (no columns: width 0)
  long long first, step;                 // of its turns

  __device__ __forceinline__ RingPlace(const RowPlan& p, uint8_t* smem, int rank) {
    data = smem + p.ring_at;
    full = smem_addr(smem) + p.bars_at;
    empty = full + 8u * p.stages;
    first = static_cast<int>(blockIdx.x) / p.ctas;
    step = static_cast<int>(gridDim.x) / p.ctas;
    col0 = rank * p.slice;
    width = max(0, min(p.slice, p.width - col0));
  }
  // One thread, before the CTA's first barrier.
  __device__ __forceinline__ void init(const RowPlan& p) const {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(full + 8u * i, p.stats_at ? 33 : 1);        // the producer's lanes, where they copy statistics
      mbar_init(empty + 8u * i, static_cast<uint32_t>(p.chunk / (p.turn / p.groups) * (p.lanes / 32)));
    }
    fence_mbar_init();
  }
};

// 4 bytes of global memory into shared memory, and this thread's arrival at a
// barrier once all such copies of its own have landed.
__device__ __forceinline__ void copy_word(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// One copy: the bytes [first, last) of a matrix, to the place in a stage that
// lies as far above a 16-byte boundary as they do.  The whole 16-byte blocks
// around them go by one bulk copy, but never from beyond the matrix: elements
// outside its whole blocks (near its two ends only) are copied here.
struct RowCopy {
  uint8_t* dst;                          // of the block that `first` lies in
  uintptr_t first, last, lo, hi;

  __device__ __forceinline__ RowCopy(const RowSource& m, uint8_t* to, uintptr_t from, uintptr_t end)
      : dst(to), first(from), last(end) {
    lo = first & ~uintptr_t{15};
    hi = (last + 15) & ~uintptr_t{15};
    if (lo < reinterpret_cast<uintptr_t>(m.p)) lo += 16;
    if (hi > reinterpret_cast<uintptr_t>(m.end)) hi -= 16;
    if (lo >= hi) lo = hi = first;
    if (lo > first || hi < last) elements(m.size);
  }
  __device__ __forceinline__ uint32_t bytes() const { return static_cast<uint32_t>(hi - lo); }
  __device__ __forceinline__ void issue(uint32_t bar) const {
    if (lo < hi)
      bulk_load(smem_addr(dst) + static_cast<uint32_t>(lo - (first & ~uintptr_t{15})),
                reinterpret_cast<const void*>(lo), bytes(), bar);
  }

 private:
  __device__ __noinline__ void elements(int size) const {
    for (uintptr_t q = first; q < last; q += size) {
      if (q >= lo && q < hi) q = hi;
      if (q >= last) break;
      uint8_t* const at = dst + (q - (first & ~uintptr_t{15}));
      if (size == 4)
        *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(q);
      else
        *reinterpret_cast<uint16_t*>(at) = *reinterpret_cast<const uint16_t*>(q);
    }
  }
};

// The work of producer warp `warp`: every plan.producers'th of the CTA's
// chunks, `stages` of all of them in flight.  A wait for a barrier's phase
// passes wrongly when the barrier is a whole phase behind, so each stage has
// one producer and the groups of one chunk: the producers and the chunks of a
// turn divide the stages, and whoever waits for a stage's phase has seen the
// phase before it.  A producer gives up at a wait that runs out (recorded), and
// in any case waits, with a limit, for its last copies: none lands in memory
// that is no longer the kernel's.  filled(): a barrier of the CTA, behind the
// first copies.
//
// Each lane has one matrix's part of a chunk (a packed one's whole, of others
// the row r; kMostChunk and kMostLoose see to it that there are enough lanes)
// and one statistic, those of stats_mask, of one of its rows.  A chunk takes a
// warp some 900 clocks (bulk copies of different lanes go one after the other):
// one producer for chunks of one row of 1024 columns made the gradient of
// 65536 of them 212 us.  Statistics that the threads loaded by themselves,
// even a row ahead, were what half of its issue slots waited for.
// ALIGNED: all rows are whole blocks.
template <bool ALIGNED, int N, class F>
__device__ __forceinline__ void produce_rows(const RowSource (&in)[N], const RowPlan& plan, const RingPlace& ring,
                                             const float* stats, uint32_t stats_mask, unsigned* err, int warp, F filled) {
  static_assert(N * kMostLoose <= 32 && kStats * kMostChunk <= 32, "a lane each");
  const int lane = threadIdx.x & 31, row_of = lane / N;
  RowSource m = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane % N == i) m = in[i];
  const bool mine = m.p && row_of < (m.packed ? 1 : plan.chunk);
  const uintptr_t base = mine ? first_byte(m, row_of, ring.col0) : 0;
  const uint32_t row_bytes = mine ? source_bytes(m.size, ring.width) : 0;
  const uint32_t more = m.packed ? m.pitch : 0;            // bytes of a further row of the chunk
  uint8_t* const to = ring.data + m.at + (m.packed ? 0u : static_cast<uint32_t>(row_of) * m.pitch);
  const bool stat = stats_mask >> (lane % kStats) & 1u;
  const float* const stat_from = stats + (lane % kStats) * plan.rows + lane / kStats;
  const uint32_t stat_to = smem_addr(ring.data) + plan.stats_at + 4u * lane;
  bool met = false;                      // the others, who fill the vectors under the first copies
  int s = 0, sub = 0;
  uint32_t ph = 0;
  long long turn = ring.first, chunk = warp;
  const auto advance = [&](int chunks) {
    for (sub += chunks * plan.chunk; sub >= plan.turn; sub -= plan.turn) turn += ring.step;
    for (s += chunks; s >= plan.stages; s -= plan.stages) ph ^= 1u;
  };
  if (warp >= plan.producers) {          // has no chunks
    filled();
    return;
  }
  advance(warp);
  for (;; chunk += plan.producers, advance(plan.producers)) {
    const long long row0 = turn * plan.turn + sub;
    if (row0 >= plan.rows) break;
    const int rows = static_cast<int>(min(static_cast<long long>(plan.chunk), plan.rows - row0));
    if (!met && chunk >= plan.stages) {
      filled();
      met = true;
    }
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(ring.empty + 8u * s, ph ^ 1u, err, kSiteProducerEmpty))) break;
    const uint32_t bar = ring.full + 8u * s, offset = static_cast<uint32_t>(s) * plan.stage_bytes;
    if (stats_mask) {                    // counted by the lanes' own arrivals
      if (stat && lane / kStats < rows) copy_word(stat_to + offset, stat_from + row0);
      copies_arrive(bar);
    }
    const bool active = mine && (m.packed || row_of < rows);
    const uintptr_t from = base + row0 * m.ld;
    const uint32_t bytes = active ? row_bytes + static_cast<uint32_t>(rows - 1) * more : 0u;
    if constexpr (ALIGNED) {
      const uint32_t whole = (bytes + 15u) & ~15u;         // 8-bit rows are padded
      const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, whole);
      if (lane == 0) mbar_arrive_expect_tx(bar, all);
      __syncwarp();
      if (whole) bulk_load(smem_addr(to) + offset, reinterpret_cast<const void*>(from), whole, bar);
    } else {
      const RowCopy copy(m, to + offset, active ? from : 0, active ? from + bytes : 0);
      const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, copy.bytes());   // behind the elements copied here
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar, all);
      __syncwarp();
      copy.issue(bar);
    }
  }
  if (!met) filled();
  __syncwarp();
  // earlier chunks than these had landed when their stages were filled again
  for (const long long last = chunk; (chunk -= plan.producers) >= 0 && chunk >= last - plan.stages;)
    mbar_wait(ring.full + 8u * static_cast<uint32_t>(chunk % plan.stages), static_cast<uint32_t>(chunk / plan.stages) & 1u, err,
              kSiteDrainTma);
}

// A computing thread's view of the ring: of its group's stages, every
// turn / chunk'th.
struct RingReader {
  const RingPlace& ring;
  const RowPlan& plan;
  unsigned* err;
  int at_row, s, step;                   // the group's first row within the stage
  uint32_t ph = 0;
  bool lost = false;

  __device__ __forceinline__ RingReader(const RingPlace& r, const RowPlan& p, unsigned* e, int first)
      : ring(r), plan(p), err(e), at_row(first % p.chunk), s(first / p.chunk), step(p.turn / p.chunk) {}
  // A wait that runs out is recorded, and the thread goes on (the result is
  // undefined, as the status says): its group's barriers need all of it.
  __device__ __forceinline__ void wait() {
    if (!lost) lost = !mbar_wait(ring.full + 8u * s, ph, err, kSiteTransformFull);
  }
  // The warp has the row in registers.
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(ring.empty + 8u * s);
    if ((s += step) >= plan.stages) {    // at least as many stages as steps
      s -= plan.stages;
      ph ^= 1u;
    }
  }
  // The statistics of the group's row i.
  __device__ __forceinline__ float4 stats(int i) const {
    return *reinterpret_cast<const float4*>(ring.data + static_cast<uint32_t>(s) * plan.stage_bytes + plan.stats_at +
                                            static_cast<uint32_t>(at_row + i) * (kStats * 4u));
  }
  // The group's row i, `row`, of a matrix in the current stage; what lies so
  // many bytes behind a 16-byte boundary in memory lies so in the stage.
  __device__ __forceinline__ const uint8_t* at(const RowSource& m, long long row, int i, bool vec) const {
    const uint8_t* const p = ring.data + static_cast<uint32_t>(s) * plan.stage_bytes + m.at +
                             static_cast<uint32_t>(at_row + i) * m.pitch;
    if (vec) return p;
    return p + (static_cast<uint32_t>(first_byte(m, m.packed ? row - at_row - i : row, ring.col0)) & 15u);
  }
};

// ---------------------------------------------------------------- a thread's part of a row
// NE elements of type T, in chunks of CP pairs.  A warp has 32 NE columns side
// by side, so that a thread's places lie a fixed distance apart, in shared and
// in global memory.  VEC: a chunk is a 16-byte vector, the warp's chunks one
// behind the other, which takes rows on 16-byte boundaries of whole vectors.
// Else single elements, 2 or 4 bytes apart from lane to lane, so that rows may
// start anywhere.
template <class T, int NE, bool VEC>
struct RowPart {
  static constexpr int V = 16 / static_cast<int>(sizeof(T));
  static constexpr int NP = NE / 2;      // pairs
  static constexpr int CP = VEC ? V / 2 : 2;
  static constexpr int NC = NP / CP;
  using Chunk = Pair[CP];
  int t, first, left;                    // column of the first element; columns from there on

  __device__ __forceinline__ RowPart(int thread, int width)
      : t(thread), first(column(thread, 0)), left(width - first) {}

  // Columns from element 0 to element i.
  static __device__ __forceinline__ constexpr int offset(int i) { return VEC ? i / V * (32 * V) + i % V : i * 32; }
  static __device__ __forceinline__ int column(int t, int i) {
    return t / 32 * (32 * NE) + t % 32 * (VEC ? V : 1) + offset(i);
  }
  __device__ __forceinline__ bool in(int i) const { return offset(i) < left; }
  __device__ __forceinline__ bool full() const { return in(NE - 1); }

  // x for pair k of chunk v, 0 for what lies outside the row.
  __device__ __forceinline__ Pair within(int v, int k, float x) const {
    const int i = VEC ? v * V : 2 * (v * CP + k);
    const float a = in(i) ? x : 0.0f;
    return pair_of(a, VEC ? a : in(i + 1) ? x : 0.0f);
  }

  // Elements of the row whose first column is at `row`; 0 for what lies outside it.
  __device__ __forceinline__ void load(const uint8_t* row, int v, Chunk& x) const {
    const T* const p = reinterpret_cast<const T*>(row) + first;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < CP; ++j) x[j] = 0;
      if (in(v * V)) pairs_of<T>(*reinterpret_cast<const uint4*>(p + offset(v * V)), x);
    } else {
#pragma unroll
      for (int j = 0; j < CP; ++j) {
        const int i = 2 * (v * CP + j);
        x[j] = pair_of(in(i) ? to_f32(p[offset(i)]) : 0.0f, in(i + 1) ? to_f32(p[offset(i + 1)]) : 0.0f);
      }
    }
  }
  // The same of a row kept in 8 bits.
  __device__ __forceinline__ void load_saved(const uint8_t* codes, const uint8_t* exponents, int v, Chunk& x) const {
    const uint8_t* const p = codes + first;
    if constexpr (VEC) {
      uint32_t w[V / 4];
      float by = 0.0f;
#pragma unroll
      for (int j = 0; j < V / 4; ++j) w[j] = 0u;
      if (in(v * V)) {
        if constexpr (V == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(p + offset(v * V));
          w[0] = q.x;
          w[V / 4 - 1] = q.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(p + offset(v * V));
        }
        by = power_of(exponents[(first + offset(v * V)) / kSavedBlock]);
      }
      const Pair power = pair_of(by, by);
#pragma unroll
      for (int j = 0; j < CP; ++j) {
        const float2 f = values_of((w[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
        x[j] = mul2(pair_of(f.x, f.y), power);
      }
    } else {
#pragma unroll
      for (int j = 0; j < CP; ++j) {
        float f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = 2 * (v * CP + j) + k;
          f[k] = in(i) ? values_of(p[offset(i)]).x * power_of(exponents[(first + offset(i)) / kSavedBlock]) : 0.0f;
        }
        x[j] = pair_of(f[0], f[1]);
      }
    }
  }
  // 0 for what lies outside the row.
  __device__ __forceinline__ void drop(int v, Pair* x) const {
    if constexpr (VEC) {
      if (!in(v * V)) {
#pragma unroll
        for (int j = 0; j < CP; ++j) x[j] = 0;
      }
    } else {
#pragma unroll
      for (int j = 0; j < CP; ++j) {
        const int i = 2 * (v * CP + j);
        float a, b;
        unpair(x[j], a, b);
        x[j] = pair_of(in(i) ? a : 0.0f, in(i + 1) ? b : 0.0f);
      }
    }
  }
  // To the row whose first column is at `row`.
  __device__ __forceinline__ void store(T* row, int v, const Chunk& x) const {
    T* const p = row + first;
    if constexpr (VEC) {
      if (in(v * V)) store_pairs(p + offset(v * V), x);
    } else {
#pragma unroll
      for (int j = 0; j < CP; ++j) {
        const int i = 2 * (v * CP + j);
        float a, b;
        unpair(x[j], a, b);
        if (in(i)) p[offset(i)] = from_f32<T>(a);
        if (in(i + 1)) p[offset(i + 1)] = from_f32<T>(b);
      }
    }
  }

  // Values per column in shared memory, laid out as the threads hold them: a
  // warp's 32 NE side by side, of these elements 4q .. 4q + 3 of its lane l at
  // 128 q + 4 l.
  static __device__ __forceinline__ int slots(int lanes) { return NE * lanes; }
  static __device__ __forceinline__ int column_of_slot(int slot) {
    const int warp = slot / (32 * NE), of = slot % (32 * NE);
    return column(warp * 32 + of % 128 / 4, of / 128 * 4 + of % 4);
  }
  __device__ __forceinline__ int slot(int q) const { return t / 32 * (32 * NE) + 128 * q + 4 * (t % 32); }
  __device__ __forceinline__ void columns(const float* values, int v, Chunk& w) const {
#pragma unroll
    for (int k = 0; k < CP / 2; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(values + slot(v * (CP / 2) + k));
      w[2 * k] = pair_of(f.x, f.y);
      w[2 * k + 1] = pair_of(f.z, f.w);
    }
  }
};

// Value c of a vector of fp32, or of T where `f32` is not set.
template <class T>
__device__ __forceinline__ float vector_value(const void* p, bool f32, long long c) {
  return f32 ? __ldg(static_cast<const float*>(p) + c) : to_f32(static_cast<const T*>(p)[c]);
}

// ---------------------------------------------------------------- sums over a row
constexpr int kMostSums = 4;             // at a time

struct RowShared {
  alignas(16) float warps[2][kRowWarps][kMostSums];        // two sets of buffers, which take turns
  float2 ctas[2][kRowWarps][kMostCtas][kMostSums / 2];     // of each group
  uint64_t bars[2][kRowWarps];
};

// Sums of N values (1, 2 or 4) over the threads of a group and, with a
// cluster, over the CTAs that share its rows; every thread gets them.  A set
// of buffers is written again only after a barrier that every reader has
// passed.  CTAs exchange theirs by asynchronous stores that a barrier at the
// destination counts, and add them in order: a barrier of the cluster would
// wait for every store in flight.
struct RowSums {
  RowShared& shared;
  const RowPlan& plan;
  unsigned* err;
  int group, t, rank;
  uint32_t flip = 0, round = 0;
  bool lost = false;

  // One thread, before the CTA's first barrier.
  static __device__ __forceinline__ void init(RowShared& shared, const RowPlan& plan) {
    for (int f = 0; f < 2; ++f)
      for (int i = 0; i < plan.groups; ++i) mbar_init(smem_addr(&shared.bars[f][i]), 1);
  }
  template <int N>
  __device__ __forceinline__ void add(float (&v)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "values");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = plan.lanes >> 5;
    // halves of the warp go on with half of the values each, until each has
    // one: value i ends up in the lanes from 32 i / N on
    float x;
    if constexpr (N == 4) {
      const bool up = lane & 16, upper = lane & 8;
      float y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) y[i] = (up ? v[N - 2 + i] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[N - 2 + i], 16);
      x = (upper ? y[1] : y[0]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? y[0] : y[1], 8);
    } else if constexpr (N == 2) {
      x = (lane < 16 ? v[0] : v[1]) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? v[1] : v[0], 16);
    } else {
      x = v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);
    }
#pragma unroll
    for (int o = N == 4 ? 4 : 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    constexpr int kLanes = 32 / N;
    if (warps > 1) {
      if (lane % kLanes == 0) shared.warps[flip][warp][lane / kLanes] = x;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(plan.lanes) : "memory");
      if (warps <= 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= warps) break;
          const float* const of = shared.warps[flip][group * warps + j];
          float f[kMostSums];
          if constexpr (N == 4)
            *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(of);
          else
            *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(of);
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] += f[i];
        }
      } else {
        // lane: value lane % N of a warp, of two with N = 4
        constexpr int kOf = N == 4 ? 8 : 16;
        const float* const of = shared.warps[flip][group * warps] + lane % N;
        const int w = lane / N % kOf;
        x = w < warps ? of[w * kMostSums] : 0.0f;
        if (N == 4 && w + kOf < warps) x += of[(w + kOf) * kMostSums];
#pragma unroll
        for (int o = N * kOf / 2; o >= N; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xFFFFFFFFu, x, i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = N == 1 ? x : __shfl_sync(0xFFFFFFFFu, x, i * kLanes);
    }
    if (plan.ctas > 1) exchange<N>(v);
    flip ^= 1u;
  }

 private:
  template <int N>
  __device__ __forceinline__ void exchange(float (&v)[N]) {
    constexpr int kPairs = (N + 1) / 2, kNext = N > 1 ? 1 : 0;
    const uint32_t bar = smem_addr(&shared.bars[flip][group]);
    if (t == 0) mbar_arrive_expect_tx(bar, plan.ctas * kPairs * 8u);
    if (t < plan.ctas) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        store_async(map_rank(smem_addr(&shared.ctas[flip][group][rank][i]), static_cast<uint32_t>(t)), v[2 * i],
                    N > 1 ? v[2 * i + kNext] : 0.0f, map_rank(bar, static_cast<uint32_t>(t)));
    }
    if (!lost) lost = !mbar_wait_cluster(bar, round, err, kSiteTransformFull);
    round ^= flip;                       // both have been waited for
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int r = 0; r < plan.ctas; ++r) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 f = shared.ctas[flip][group][r][i];
        v[2 * i] += f.x;
        if (N > 1) v[2 * i + kNext] += f.y;
      }
    }
  }
};

}  // namespace
}  // namespace gemm_f32_impl
