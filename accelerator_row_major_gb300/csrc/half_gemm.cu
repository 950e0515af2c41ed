// bfloat16 tensor-core product on CTA pairs (tcgen05 cta_group::2) for
// sm_103a: D = A B^T with fp32 accumulation, stored scaled, or reduced to
// the softmax statistics of its rows without being stored.
//
// A tile of 256 x 256 is computed by a cluster of two CTAs on two SMs: CTA r
// holds rows 128 r .. +127 of the A tile and of the B tile in shared memory
// and the accumulator of its 128 rows of D by all 256 columns in tensor
// memory; one M = 256 MMA issued by the even CTA works on both.  Every
// operand byte a CTA loads feeds 256 multiply-adds, half the loads of a
// 128 x 256 tile per CTA.  Operands come by TMA in 128-byte swizzled slices
// 64 deep along K, K-major or MN-major as they are stored (the MMA reads
// either, so nothing is ever transposed), five stages of 32 KB in flight.
// The accumulator is double buffered (2 x 256 of the 512 columns of tensor
// memory), so a tile's epilogue runs under the next tile's MMAs.
//
// Roles per CTA (384 threads): warp 0 TMA producer (its own halves; both
// CTAs' bytes are counted on the even CTA's barrier), warp 1 tensor memory
// and, in the even CTA, the MMAs; warps 4 .. 11 epilogue: four warps for
// each half of the columns, one row of D per thread and half.
//
// fp32 operands (PARTS = 3): each is the sum of three bfloat16 parts, hi +
// mid + lo, 24 significant bits.  Of the nine products the six that reach
// fp32's precision are taken: lo hi, hi lo, mid mid, mid hi, hi mid, hi hi
// (the dropped ones are below 2^-24 of the product).  The tensor core adds
// into its accumulator by truncation (measured: a sum over K drifts towards
// zero by about 1e-9 K of its size), so the accumulator takes only 256 of K
// at a time, smallest products first, and the epilogue warps add these
// partial sums in registers, rounding to nearest.  With a right operand that
// is bfloat16 as it is (PARTS = kLeftParts) three products do: lo, mid, hi.
//
// Work: whole tiles round robin over the pairs; the tiles of the last,
// partial wave are split along K over all pairs, whose partial tiles a
// second kernel adds in order.  Four pairs (two, where the numbers divide by
// no more) form a team that walks the same K range of four neighbouring
// tiles, two by two where all tiles are split, so that the operands the
// tiles share are in the L2 when the others want them: alone, each pair would
// read its own range of them at its own time (gradients of 4096 x 1024 x
// 32768 fp32 3007 us against 2895, 8192 x 1024 x 65536 bfloat16 2439 against
// 2319, a few calls in a row; at the clocks of calls without end the former
// takes 3.2 ms).  Logits are not split (their epilogue needs
// the whole sum).  Every wait is bounded, as in the library's other kernels.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/gemm_f32.h"
#include "device_common.cuh"
#include "half_gemm.h"
#include "launch.h"
#include "pair_common.cuh"
#include "row_common.cuh"

namespace gemm_f32_impl {
using namespace gemm_f32_dev;

namespace {

constexpr int kHalf = 128;               // rows of A and of B per CTA
constexpr int kTile = 256;
constexpr int kBK = 64;                  // 128 bytes of K per stage
constexpr int kStages = 5;
constexpr int kOperandBytes = kHalf * kBK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStagingBytes = 4096;      // 32 rows of 128 bytes; two per epilogue warp
constexpr int kStagingBuffers = 2;
constexpr int kThreads = 384;
constexpr int kEpilogueWarp0 = 4;
constexpr int kEpilogueWarps = 8;
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStagingBuffers * kStagingBytes + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");
constexpr int kTmemCols = 512;
constexpr int kRasterGroup = 8;
constexpr int kSplitRaster = 2;          // where all tiles are split
constexpr int kMinSplitBlocks = 16;      // least K blocks per pair in the split tail
constexpr int kMostTeam = 4;
// K blocks that one accumulator sums before its sum goes on in registers:
// 256 of K for fp32 operands, and 1024 for the logits of bfloat16 ones, and
// their products that ask for it, where a pair has more of a tile than that
// (0: all of it).
constexpr int kSumF32 = 4;
constexpr int kSumHalf = 16;
constexpr int kLeftParts = 2;            // PARTS: the left operand alone comes in three

// Epilogues
constexpr int kLogits = 0;
constexpr int kStoreBf16 = 1;
constexpr int kStoreF32 = 2;

struct Params {
  int M, N;
  int tiles_m, tiles_n;
  int k_blocks;                          // of 64
  int k_iters;                           // units of the work list: blocks, or sums of SUM blocks
  int raster;                            // rows of tiles that are walked together
  int team;                              // pairs that share K ranges of the split tiles
  int dp_tiles, sk_ctas, max_seg;        // sk_ctas: teams
  long long sk_work;                     // of the teams
  float* partials;                       // [tail][max_seg][256][256]
  void* c;
  long long ldc;
  int c_f32;
  int c_tma;                             // TMA can write C (tmC), else stores of single elements
  const float* scale;
  const float* add;
  long long ldadd;
  int add_vec;                           // rows of `add` take 16-byte loads
  float2* stats;
  long long ld_stats;
  void* exps;
  long long ld_exps;
  LossTargets targets;
  float* label_logit;
  unsigned* arrived;
  unsigned* err;
};

// ---------------------------------------------------------------- primitives
// 3-D tiled copy into this CTA's shared memory whose bytes are counted on a
// barrier of either CTA of the pair (a shared::cluster address).  The inner
// coordinate x is a multiple of 64 elements (128 bytes).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* desc, uint32_t bar, int x,
                                              int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(desc), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 2-D tiled copy of 32 rows of 128 bytes out of shared memory; columns and
// rows outside the map are not written.
__device__ __forceinline__ void tma_store(const void* desc, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(desc),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All but this thread's latest group of stores have read their shared memory
// / all have been made.
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16, bfloat16 operands, fp32 accumulator
// (fields as idesc_tf32; format 1 = bfloat16).
constexpr uint32_t idesc_bf16(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(n) >> 3) << 17) | ((static_cast<uint32_t>(m) >> 4) << 24);
}

// Descriptor of the 16-deep K slice kk of a staged operand of 128 x 64.
// K-major: 128 rows of 128 bytes, eight rows per swizzle atom (stride 1024);
// slice kk starts 32 bytes further in the row.  MN-major: two chunks (8 KB
// apart, the leading offset) of 64 K rows of 64 MN elements, eight K rows
// per atom (stride 1024); slice kk starts 16 rows further.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, int kk) {
  return MN ? smem_desc(addr + kk * 2048, 8192, 1024, 2) : smem_desc(addr + kk * 32, 16, 1024, 2);
}

struct PairItems {
  int member, team, units, next_dp;
  long long x, x_end;

  __device__ __forceinline__ explicit PairItems(const Params& p) {
    next_dp = static_cast<int>(blockIdx.x >> 1);
    units = static_cast<int>(gridDim.x >> 1);
    team = next_dp / p.team;
    member = next_dp % p.team;
    x = x_end = 0;
    if (team < p.sk_ctas) {
      x = sk_start(team, p.sk_ctas, p.sk_work);
      x_end = sk_start(team + 1, p.sk_ctas, p.sk_work);
    }
  }

  __device__ __forceinline__ bool next(const Params& p, WorkItem& w) {
    if (next_dp < p.dp_tiles) {
      w.tile = next_dp;
      w.k0 = 0;
      w.k1 = p.k_iters;
      w.tail = -1;
      w.seg = 0;
      w.nseg = 1;
      next_dp += units;
      return true;
    }
    if (x >= x_end) return false;
    const long long ki = p.k_iters;
    const int i = static_cast<int>(x / ki);
    w.tail = i * p.team + member;
    w.tile = p.dp_tiles + w.tail;
    w.k0 = static_cast<int>(x - i * ki);
    w.k1 = static_cast<int>(min(ki, w.k0 + (x_end - x)));
    const int first = sk_owner(i * ki, p.sk_ctas, p.sk_work);
    w.seg = team - first;
    w.nseg = sk_owner((i + 1) * ki - 1, p.sk_ctas, p.sk_work) - first + 1;
    x += w.k1 - w.k0;
    return true;
  }
};

// Elements of the partial tiles, for the checked build.
[[maybe_unused]] __device__ __forceinline__ size_t partials_extent(const Params& p) {
  return static_cast<size_t>(p.tiles_m * p.tiles_n - p.dp_tiles) * p.max_seg * (kTile * kTile);
}

// The sums of NC consecutive columns of one row of C, scaled and added to.
template <int NC>
__device__ __forceinline__ void finish_c(const Params& p, int row, int col, float s, float (&v)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) v[j] *= s;
  if (p.add == nullptr || row >= p.M) return;
  const float* const add = p.add + static_cast<size_t>(row) * p.ldadd + col;
  if (p.add_vec && col + NC <= p.N) {
#pragma unroll
    for (int j = 0; j < NC / 4; ++j) {
      const float4 a = reinterpret_cast<const float4*>(add)[j];
      v[4 * j] += a.x;
      v[4 * j + 1] += a.y;
      v[4 * j + 2] += a.z;
      v[4 * j + 3] += a.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (col + j < p.N) v[j] += add[j];
  }
}

// Columns from `valid` on become -inf (a power of 0).
__device__ __forceinline__ void mask_columns(float (&v)[32], int valid) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = j < valid ? v[j] : -INFINITY;
}

// 16-byte chunk c of row r of a staging buffer (32 rows of 128 bytes in the
// 128-byte swizzle that TMA undoes).
__device__ __forceinline__ uint32_t staged(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// Two values as bfloat16 or fp16, or chunks of them.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_fp16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// This lane's row of 32 values into its staging buffer: a whole row of 32
// fp32 values, or half (0, 1) of a row of 64 16-bit ones.
__device__ __forceinline__ void stage_f32(uint8_t* buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(buf + staged(lane, c)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
template <bool FP16>
__device__ __forceinline__ void stage_16(uint8_t* buf, int lane, int half, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = FP16 ? pack_fp16(v[8 * c + 2 * j], v[8 * c + 2 * j + 1])
                  : pack_bf16(v[8 * c + 2 * j], v[8 * c + 2 * j + 1]);
    *reinterpret_cast<uint4*>(buf + staged(lane, 4 * half + c)) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// Writes a staged block to C rows row0 .., columns col0 ..: one TMA store,
// or, where TMA cannot address C, one row after the other with the lanes
// along the columns.
template <class T>
__device__ __forceinline__ void write_staged(const Params& p, const void* tmC, const uint8_t* buf,
                                             int lane, int row0, int col0) {
  constexpr int kCols = 128 / static_cast<int>(sizeof(T)), kPer = 16 / static_cast<int>(sizeof(T));
  const bool any = row0 < p.M && col0 < p.N;
  if (p.c_tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (any) tma_store(tmC, smem_addr(buf), col0, row0);
      tma_store_commit();   // one group per block, empty or not: the waits count groups
    }
    return;
  }
  if (!any) return;
  __syncwarp();
  T* const c = static_cast<T*>(p.c);
  const int rows = min(32, p.M - row0);
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int j = lane; j < kCols; j += 32) {
      const size_t at = static_cast<size_t>(row0 + r) * p.ldc + col0 + j;
      if (col0 + j < p.N && GEMM_IN_EXTENT(at, stored_extent(p.M, p.N, p.ldc), p.err, kSiteBoundsC))
        c[at] = *reinterpret_cast<const T*>(buf + staged(r, j / kPer) + (j % kPer) * sizeof(T));
    }
}

// ---------------------------------------------------------------- kernel
template <bool A_MN, bool B_MN, int PARTS, int SUM, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    half_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr int S = kStages;
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t dyn0 = smem_addr(smem_dyn);
  const uint32_t base = (dyn0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_dyn + (base - dyn0);
  uint8_t* const staging = base_ptr + S * kStageBytes;
  const uint32_t bars = base + S * kStageBytes + kEpilogueWarps * kStagingBuffers * kStagingBytes;
  auto full_bar = [&](int s) { return bars + 8u * s; };          // both CTAs' bytes (even CTA's)
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };   // MMAs done with the stage
  auto accf_bar = [&](int b) { return bars + 8u * (2 * S + b); };      // accumulator complete
  auto acce_bar = [&](int b) { return bars + 8u * (2 * S + 2 + b); };  // drained (even CTA's)
  const uint32_t drain_bar = bars + 8u * (2 * S + 4);
  const uint32_t tmem_slot = bars + 8u * (2 * S + 5);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);   // warp-uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * kEpilogueWarps);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();      // barriers of both CTAs exist before any remote arrive
  tc_fence_after_sync();
  const uint32_t tmem_base = __shfl_sync(
      0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(base_ptr + (tmem_slot - base)), 0);
  grid_launch_dependents();
  grid_dependency_wait();   // global memory from here on
  if (EPI == kLogits && blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0u;

  // K blocks of unit u of the work list, and how often they are passed over
  constexpr int kCombos = PARTS == 3 ? 6 : PARTS == kLeftParts ? 3 : 1;
  auto first_block = [&](int u) { return SUM ? u * SUM : u; };
  auto end_block = [&](int u) { return SUM ? min((u + 1) * SUM, p.k_blocks) : u + 1; };

  WorkItem w;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (own halves)
    if (lane == 0) {
      const uint32_t leader_full0 = map_rank(full_bar(0), 0);
      int s = 0;
      uint32_t ph = 0, armed = 0, last_ph = 0;
      bool ok = true;
      PairItems list(p);
      while (ok && list.next(p, w)) {
        const TileCoord c = tile_coord(w.tile, p.tiles_m, p.tiles_n, p.raster, true);
        const int m0 = c.tm * kTile + static_cast<int>(rank) * kHalf;
        const int n0 = c.tn * kTile + static_cast<int>(rank) * kHalf;
        for (int u = w.k0; ok && u < w.k1; ++u) {
          for (int combo = 0; ok && combo < kCombos; ++combo) {
            // (lo, hi), (hi, lo), (mid, mid), (mid, hi), (hi, mid), (hi, hi)
            const int pa = PARTS == 3 ? (0x001102 >> (4 * combo)) & 3 : PARTS == kLeftParts ? 2 - combo : 0;
            const int pb = PARTS == 3 ? (0x010120 >> (4 * combo)) & 3 : 0;
            for (int kb = first_block(u); kb < end_block(u); ++kb) {
              if (!mbar_wait(empty_bar(s), ph ^ 1u, p.err, kSiteProducerEmpty)) {
                ok = false;
                break;
              }
              const uint32_t st = base + s * kStageBytes;
              const uint32_t bar = leader_full0 + 8u * s;
              if (rank == 0) {
                mbar_arrive_expect_tx(full_bar(s), 2 * kStageBytes);
                armed |= 1u << s;
                last_ph = (last_ph & ~(1u << s)) | (ph << s);
              }
              const int k = kb * kBK;
              if (A_MN) {
                tma_load_pair(st, &tmA, bar, m0, k, pa);
                tma_load_pair(st + 8192, &tmA, bar, m0 + 64, k, pa);
              } else {
                tma_load_pair(st, &tmA, bar, k, m0, pa);
              }
              if (B_MN) {
                tma_load_pair(st + kOperandBytes, &tmB, bar, n0, k, pb);
                tma_load_pair(st + kOperandBytes + 8192, &tmB, bar, n0 + 64, k, pb);
              } else {
                tma_load_pair(st + kOperandBytes, &tmB, bar, k, n0, pb);
              }
              if (++s == S) {
                s = 0;
                ph ^= 1u;
              }
            }
          }
        }
      }
      // both CTAs' copies have landed before either CTA's memory goes away
      for (int q = 0; q < S; ++q)
        if (armed & (1u << q)) mbar_wait(full_bar(q), (last_ph >> q) & 1u, p.err, kSiteDrainTma);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16(2 * kHalf, kTile, A_MN, B_MN);
      const bool issuer = elect_lane();
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      // One accumulator's sum: over the whole item, or over one unit of it.
      auto open = [&]() {
        const bool got = mbar_wait_cluster(acce_bar(buf), acc_ph ^ 1u, p.err, kSiteMmaAccEmpty);
        tc_fence_after_sync();
        return __all_sync(0xFFFFFFFFu, got) != 0;
      };
      auto close = [&]() {
        if (issuer) mma_commit_both(accf_bar(buf));
        __syncwarp();
        buf ^= 1;
        if (buf == 0) acc_ph ^= 1u;
      };
      PairItems list(p);
      while (ok && list.next(p, w)) {
        uint32_t more = 0;
        if (!SUM && !open()) break;
        for (int u = w.k0; ok && u < w.k1; ++u) {
          if (SUM) {
            more = 0;
            if (!open()) {
              ok = false;
              break;
            }
          }
          const int blocks = kCombos * (end_block(u) - first_block(u));
          for (int i = 0; i < blocks; ++i) {
            const bool got = mbar_wait_cluster(full_bar(s), ph, p.err, kSiteMmaReady);
            if (!__all_sync(0xFFFFFFFFu, got)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t st = base + s * kStageBytes;
            const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * kTile);
            if (issuer) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                mma_bf16_pair(acc, operand_desc<A_MN>(st, kk),
                              operand_desc<B_MN>(st + kOperandBytes, kk), idesc, kk ? 1u : more);
              mma_commit_both(empty_bar(s));
            }
            __syncwarp();
            more = 1u;
            if (++s == S) {
              s = 0;
              ph ^= 1u;
            }
          }
          if (SUM && ok) close();
        }
        if (!SUM && ok) close();
      }
      if (issuer) {
        mma_commit_local(drain_bar);
        mbar_wait(drain_bar, 0, p.err, kSiteDrainMma);
      }
    }
    __syncwarp();
  } else if (warp >= kEpilogueWarp0) {
    // ------------------------------------------------------------ epilogue (own rows)
    const int q = warp & 3;                                    // 32 lanes of tensor memory
    const int half = (warp - kEpilogueWarp0) >> 2;             // 128 of the 256 columns
    const uint32_t t_mine =
        tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kHalf);
    const uint32_t leader_acce0 = map_rank(acce_bar(0), 0);
    int buf = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    auto wait_full = [&]() {
      const bool got = mbar_wait(accf_bar(buf), acc_ph, p.err, kSiteEpilogueFull);
      tc_fence_after_sync();
      return __all_sync(0xFFFFFFFFu, got) != 0;
    };
    auto release = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(leader_acce0 + 8u * buf);
      buf ^= 1;
      if (buf == 0) acc_ph ^= 1u;
    };
    uint8_t* const stages = staging + (warp - kEpilogueWarp0) * (kStagingBuffers * kStagingBytes);
    uint8_t* stage = stages;
    auto stage_free = [&]() {   // on to the other buffer, whose last store has read it
      stage = stage == stages ? stages + kStagingBytes : stages;
      if (lane == 0) tma_store_wait_read();
      __syncwarp();
    };
    [[maybe_unused]] const float scale = p.scale ? __ldg(p.scale) : 1.0f;
    PairItems list(p);
    while (ok && list.next(p, w)) {
      const TileCoord c = tile_coord(w.tile, p.tiles_m, p.tiles_n, p.raster, true);
      const int local = static_cast<int>(rank) * kHalf + q * 32 + lane;
      const int row = c.tm * kTile + local;
      const int n0 = c.tn * kTile + half * kHalf;
      [[maybe_unused]] float acc[SUM ? kHalf : 1];
      if constexpr (SUM != 0) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) acc[j] = 0.0f;
        for (int u = w.k0; u < w.k1; ++u) {
          if (!wait_full()) {
            ok = false;
            break;
          }
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t v[32];
            tmem_ld_32cols(t_mine + static_cast<uint32_t>(buf * kTile + ch * 32), v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[ch * 32 + j] += __uint_as_float(v[j]);
          }
          release();
        }
        if (!ok) break;
      } else {
        if (!wait_full()) break;
      }
      // 32 columns of this thread's row; the last load frees the accumulator
      auto take = [&](int ch, float(&v)[32], bool last) {
        if constexpr (SUM != 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = acc[ch * 32 + j];
        } else {
          uint32_t u[32];
          tmem_ld_32cols(t_mine + static_cast<uint32_t>(buf * kTile + ch * 32), u);
          tmem_wait_ld();
          if (last) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
        }
      };
      if constexpr (EPI != kLogits) {
        if (w.nseg > 1) {
          float* const part = p.partials +
                              (static_cast<size_t>(w.tail) * p.max_seg + w.seg) * (kTile * kTile) +
                              static_cast<size_t>(local) * kTile + half * kHalf;
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            float v[32];
            take(ch, v, ch == 3);
            if (GEMM_IN_EXTENT(part + ch * 32 + 31 - p.partials, partials_extent(p), p.err, kSiteBoundsWork))
              store_vec<float, 32>(part + ch * 32, v);
          }
        } else {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            float v[32];
            take(ch, v, ch == 3);
            finish_c<32>(p, row, n0 + ch * 32, scale, v);
            if (EPI == kStoreF32 || ch % 2 == 0) stage_free();
            if constexpr (EPI == kStoreF32) {
              stage_f32(stage, lane, v);
              write_staged<float>(p, &tmC, stage, lane, row - lane, n0 + ch * 32);
            } else {
              stage_16<false>(stage, lane, ch % 2, v);
              if (ch % 2)
                write_staged<__nv_bfloat16>(p, &tmC, stage, lane, row - lane, n0 + (ch - 1) * 32);
            }
          }
        }
      } else {
        const bool row_ok = row < p.M;
        const bool whole = n0 + kHalf <= p.N;      // else columns from N on are masked
        float top = -INFINITY;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float v[32];
          take(ch, v, false);
          if (!whole) mask_columns(v, p.N - n0 - ch * 32);
          float t[4] = {v[0], v[1], v[2], v[3]};   // four chains
#pragma unroll
          for (int j = 4; j < 32; ++j) t[j % 4] = fmaxf(t[j % 4], v[j]);
          top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])));
        }
        const float below = -reference(top);
        const int label = row_ok ? label_at(p.targets, row) - n0 : -1;
        // one part: powers times 2^15, which keep their 11 bits in fp16 down to 2^-29
        constexpr float kUp = PARTS == 3 ? 0.0f : 15.0f;
        const Pair minus = pair_of(below, below), by = pair_of(kLog2e, kLog2e), up = pair_of(kUp, kUp);
        Pair sums = 0;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float v[32];
          take(ch, v, ch == 3);
          if (!whole) mask_columns(v, p.N - n0 - ch * 32);
          if (__any_sync(0xFFFFFFFFu, label >= ch * 32 && label < ch * 32 + 32)) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = label == ch * 32 + j ? v[j] : z;
            if (label >= ch * 32 && label < ch * 32 + 32) p.label_logit[row] = z;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            unpair(fma2(add2(pair_of(v[j], v[j + 1]), minus), by, up), v[j], v[j + 1]);
            v[j] = exp2_approx(v[j]);
            v[j + 1] = exp2_approx(v[j + 1]);
            sums = add2(sums, pair_of(v[j], v[j + 1]));
          }
          if (p.exps) {   // C is the matrix of exponentials: fp32, or fp16
            if (PARTS == 3 || ch % 2 == 0) stage_free();
            if constexpr (PARTS == 3) {
              stage_f32(stage, lane, v);
              write_staged<float>(p, &tmC, stage, lane, row - lane, n0 + ch * 32);
            } else {
              stage_16<true>(stage, lane, ch % 2, v);
              if (ch % 2) write_staged<__half>(p, &tmC, stage, lane, row - lane, n0 + (ch - 1) * 32);
            }
          }
        }
        const size_t stat = static_cast<size_t>(2 * c.tn + half) * p.ld_stats + row;
        if (row_ok && GEMM_IN_EXTENT(stat, 2 * static_cast<size_t>(p.tiles_n) * p.ld_stats, p.err,
                                     kSiteBoundsScratch))
          p.stats[stat] =
              make_float2(top, PARTS == 3 ? sum_of(sums) : sum_of(sums) * (1.0f / 32768.0f));
      }
    }
    if (lane == 0) tma_store_wait();
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();   // the even CTA's MMAs and both CTAs' copies have finished
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// C of the split tiles: each tile's partials added in segment order.  One
// CTA per 4 rows of a tile, 4 columns per thread.
__global__ void __launch_bounds__(256) half_gemm_reduce_kernel(const Params p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int tail = blockIdx.x / 64;
  const int local = (blockIdx.x % 64) * 4 + threadIdx.x / 64;
  const int col = (threadIdx.x % 64) * 4;
  const long long ki = p.k_iters;
  const int shared = tail / p.team;       // the team's tiles have their K ranges in common
  const int nseg = sk_owner((shared + 1) * ki - 1, p.sk_ctas, p.sk_work) -
                   sk_owner(shared * ki, p.sk_ctas, p.sk_work) + 1;
  if (nseg == 1) return;   // its one pair stored it
  const TileCoord c = tile_coord(p.dp_tiles + tail, p.tiles_m, p.tiles_n, p.raster, true);
  const int row = c.tm * kTile + local, n = c.tn * kTile + col;
  if (row >= p.M || n >= p.N) return;
  const float* src = p.partials + static_cast<size_t>(tail) * p.max_seg * (kTile * kTile) +
                     static_cast<size_t>(local) * kTile + col;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < nseg; ++s, src += kTile * kTile) {
    if (!GEMM_IN_EXTENT(src + 3 - p.partials, partials_extent(p), p.err, kSiteBoundsWork)) return;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
    v[0] += x.x;
    v[1] += x.y;
    v[2] += x.z;
    v[3] += x.w;
  }
  finish_c<4>(p, row, n, p.scale ? __ldg(p.scale) : 1.0f, v);
  const size_t at = static_cast<size_t>(row) * p.ldc + n;
  if (p.c_tma && n + 4 <= p.N) {   // rows on 16-byte boundaries
    if (!GEMM_IN_EXTENT(at + 3, stored_extent(p.M, p.N, p.ldc), p.err, kSiteBoundsC)) return;
    if (p.c_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.c) + at) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n + j >= p.N || !GEMM_IN_EXTENT(at + j, stored_extent(p.M, p.N, p.ldc), p.err, kSiteBoundsC))
      continue;
    if (p.c_f32)
      static_cast<float*>(p.c)[at + j] = v[j];
    else
      static_cast<__nv_bfloat16*>(p.c)[at + j] = __float2bfloat16_rn(v[j]);
  }
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

int blocks_of(int n, int per) { return (n - 1) / per + 1; }

// Tiles, K units and the split of the last wave; returns the bytes of
// partial tiles.
size_t plan_tiles(Params& p, int M, int N, int K, int sum, int num_sms, bool split) {
  p.M = M;
  p.N = N;
  p.tiles_m = blocks_of(M, kTile);
  p.tiles_n = blocks_of(N, kTile);
  p.k_blocks = blocks_of(K, kBK);
  p.k_iters = sum ? blocks_of(p.k_blocks, sum) : p.k_blocks;
  const long tiles = static_cast<long>(p.tiles_m) * p.tiles_n;
  p.dp_tiles = static_cast<int>(tiles);
  p.sk_ctas = 0;
  p.sk_work = 0;
  p.max_seg = 1;
  p.raster = kRasterGroup;
  p.team = 1;
  if (!split) return 0;
  const int pairs = num_sms / 2;
  const long tail = tiles % pairs;
  for (int team = kMostTeam; team > 1 && p.team == 1; team /= 2)
    if (pairs % team == 0 && tail % team == 0) p.team = team;
  const size_t bytes = plan_split_tail(p, tiles / p.team, pairs / p.team, sizeof(float) * kTile * kTile * p.team,
                                       sum ? 1 : kMinSplitBlocks);
  p.dp_tiles = bytes ? p.dp_tiles * p.team : static_cast<int>(tiles);
  if (p.dp_tiles == 0) p.raster = kSplitRaster;
  return bytes;
}

// The same, and the K blocks that one accumulator sums.
enum Product { kLogitsOf, kStored, kSummed };
size_t plan(Params& p, int M, int N, int K, int parts, Product product, int num_sms, int* sum) {
  const bool split = product != kLogitsOf;
  *sum = parts == 3 ? kSumF32 : 0;
  const size_t bytes = plan_tiles(p, M, N, K, *sum, num_sms, split);
  if (parts == 3 || product == kStored) return bytes;
  // the most that a pair has of one tile: in units of 1024 of K the work splits less finely (2048 x 1024 x 1024 bfloat16
  // 22.3 us against 21.4 with as little as that of a tile anyway, 65536 x 256 x 256 52 against 35)
  const long long most = p.dp_tiles > 0 || p.sk_ctas == 0 ? p.k_blocks : (p.sk_work - 1) / p.sk_ctas + 1;
  if (most <= kSumHalf) return bytes;
  *sum = kSumHalf;
  return plan_tiles(p, M, N, K, *sum, num_sms, split);
}

// 2-D map of what the epilogue writes (rows on 16-byte boundaries): boxes of
// 32 rows of 128 bytes.
bool encode_c(CUtensorMap* map, const void* c, long long ldc, int rows, long long cols,
              CUtensorMapDataType type, int size) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tma_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldc) * size};
  const cuuint32_t box[2] = {128u / size, 32u};
  const cuuint32_t step[2] = {1u, 1u};
  return enc(map, type, 2, const_cast<void*>(c), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [parts][rows][cols] bfloat16, box of 64 columns by box_rows rows of one part.
bool encode(CUtensorMap* map, const HalfOperand& o, int rows, int cols, int parts, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tma_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(o.ld) * 2u;
  const cuuint64_t strides[2] = {
      row_bytes, parts > 1 ? static_cast<cuuint64_t>(o.plane) * 2u : row_bytes * dims[1]};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.ptr), dims, strides, box,
             step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap a, b, c;
};

template <bool A_MN, bool B_MN, int PARTS, int SUM, int EPI>
int launch_one(const HalfGemm& g, const Params& p, const Maps& m, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};   // bit per device
  auto kern = half_gemm_kernel<A_MN, B_MN, PARTS, SUM, EPI>;
  const unsigned long long bit = 1ull << (g.device % kMaxDevices);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    configured.fetch_or(bit);
  }
  if (launch_dependent(kern, dim3(grid), dim3(kThreads), kSmem, stream, m.a, m.b, m.c, p) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

// The forms the vocabulary loss and the weight gradient need: logits of
// K-major operands, and products with an MN-major right operand.
int launch_form(const HalfGemm& g, const Params& p, const Maps& m, int sum, int grid, cudaStream_t stream) {
  if (!g.c) {
    if (g.parts == 3) return launch_one<false, false, 3, kSumF32, kLogits>(g, p, m, grid, stream);
    if (sum) return launch_one<false, false, 1, kSumHalf, kLogits>(g, p, m, grid, stream);
    return launch_one<false, false, 1, 0, kLogits>(g, p, m, grid, stream);
  }
  if (g.parts == 3) {
    if (!g.c_f32 || (g.b_whole && !g.a.mn_major)) return GEMM_F32_EINVAL;
    if (g.b_whole) return launch_one<true, true, kLeftParts, kSumF32, kStoreF32>(g, p, m, grid, stream);
    return g.a.mn_major ? launch_one<true, true, 3, kSumF32, kStoreF32>(g, p, m, grid, stream)
                        : launch_one<false, true, 3, kSumF32, kStoreF32>(g, p, m, grid, stream);
  }
  if (g.c_f32) {
    if (!g.a.mn_major) return GEMM_F32_EINVAL;
    return sum ? launch_one<true, true, 1, kSumHalf, kStoreF32>(g, p, m, grid, stream)
               : launch_one<true, true, 1, 0, kStoreF32>(g, p, m, grid, stream);
  }
  if (sum && !g.a.mn_major) return GEMM_F32_EINVAL;
  if (sum) return launch_one<true, true, 1, kSumHalf, kStoreBf16>(g, p, m, grid, stream);
  return g.a.mn_major ? launch_one<true, true, 1, 0, kStoreBf16>(g, p, m, grid, stream)
                      : launch_one<false, true, 1, 0, kStoreBf16>(g, p, m, grid, stream);
}

}  // namespace

size_t half_gemm_scratch(int M, int N, int K, int parts, int num_sms, bool summed) {
  Params p = {};
  int sum = 0;
  return plan(p, M, N, K, parts, summed ? kSummed : kStored, num_sms, &sum);
}

int launch_half_gemm(const HalfGemm& g, cudaStream_t stream, int* launches) {
  const int pairs = g.num_sms / 2;
  if (pairs < 1) return GEMM_F32_EDEVICE;
  if (g.c ? !g.b.mn_major : g.a.mn_major || g.b.mn_major) return GEMM_F32_EINVAL;
  Params p = {};
  int sum = 0;
  plan(p, g.M, g.N, g.K, g.parts, !g.c ? kLogitsOf : g.summed ? kSummed : kStored, g.num_sms, &sum);
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x7fffffffLL) return GEMM_F32_EINVAL;
  p.partials = g.partials;
  p.c = g.c;
  p.ldc = g.ldc;
  p.c_f32 = g.c_f32;
  p.scale = g.scale;
  p.add = g.add;
  p.ldadd = g.ldadd;
  p.add_vec = reinterpret_cast<uintptr_t>(g.add) % 16 == 0 && g.ldadd % 4 == 0;
  p.stats = g.stats;
  p.ld_stats = g.ld_stats;
  p.exps = g.exps;
  p.ld_exps = g.ld_exps;
  p.targets = g.targets;
  p.label_logit = g.label_logit;
  p.arrived = g.arrived;
  p.err = g.err;
  Maps m = {};
  const int b_parts = g.b_whole ? 1 : g.parts;
  if (!(g.a.mn_major ? encode(&m.a, g.a, g.K, g.M, g.parts, 64)
                     : encode(&m.a, g.a, g.M, g.K, g.parts, kHalf)) ||
      !(g.b.mn_major ? encode(&m.b, g.b, g.K, g.N, b_parts, 64)
                     : encode(&m.b, g.b, g.N, g.K, b_parts, kHalf)))
    return GEMM_F32_ELAUNCH;
  if (g.c) {
    const int size = g.c_f32 ? 4 : 2;
    p.c_tma = reinterpret_cast<uintptr_t>(g.c) % 16 == 0 && g.ldc * size % 16 == 0 &&
              encode_c(&m.c, g.c, g.ldc, g.M, g.N,
                       g.c_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, size);
  } else if (g.exps) {   // all ceil(N / 256) 256 columns
    const bool f32 = g.parts == 3;
    if (!encode_c(&m.c, g.exps, g.ld_exps, g.M, g.ld_exps,
                  f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, f32 ? 4 : 2))
      return GEMM_F32_ELAUNCH;
    p.c_tma = 1;
  }
  const int units = p.sk_ctas > 0 ? pairs : static_cast<int>(std::min<long long>(tiles, pairs));
  const int rc = launch_form(g, p, m, sum, 2 * units, stream);
  if (rc != GEMM_F32_OK) return rc;
  ++*launches;
  if (p.sk_ctas > 0) {
    const unsigned tail = static_cast<unsigned>(tiles - p.dp_tiles);
    if (launch_dependent(half_gemm_reduce_kernel, dim3(tail * 64), dim3(256), 0, stream, p) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    ++*launches;
  }
  return GEMM_F32_OK;
}

}  // namespace gemm_f32_impl
