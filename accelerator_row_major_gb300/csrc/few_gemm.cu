// The vocabulary loss's products for few rows (sm_103a): with T <= 128 rows
// the logits z = x w^T and dx = g w are bound by the one read of w, so here w
// is the operand along M (128 of its rows, or columns, per tile) and the rows
// are the MMA's N (T rounded up to 16), one CTA per SM.
//
//   logits  D[v][t] = sum_d w[v][d] x[t][d]: A = w, K-major.  Each CTA takes
//           an even share of w's rows (in units of 32), in tiles of up to 128.
//           TMA reads rows whose distance is a multiple of 16 bytes from a
//           16-byte boundary on.  Where w's own are not (an odd width), every
//           8th (or 4th, 2nd) row has the same distance from a boundary, so
//           these classes of rows are read as matrices of their own, from the
//           boundary below: the elements in front of a row become zeros in
//           the tile, and x is there once for each class, shifted alike.
//   dx      D[d][t] = sum_v w[v][d] g[t][v]: A = w^T, MN-major.  Tiles of 128
//           columns; their K (the vocabulary) is shared evenly by all CTAs,
//           and a second kernel adds the partial tiles in order.
//
// bfloat16: w's tiles go from TMA to the MMA as they are.  fp32 (F32): w is
// never stored in parts; eight warps read each landed tile of 128 x 64, split
// every value into hi + mid + lo (24 bits) and write the parts to tensor
// memory, where the MMA takes its A operand.  The six products of half_gemm.cu
// are summed for a stretch of K and the sums are added in registers to
// nearest, since the tensor core's own additions truncate.  Up to 64 rows the
// parts of b lie one below the other as one operand of 3 n, so three MMAs
// make the six products, [hi | mid | lo] by hi, [hi | mid] by mid, [hi] by
// lo, into three accumulators by size, each 512 of K long (an MMA was
// measured to cost n / 2 + 26 clocks); above, tensor memory has no room for
// them and six MMAs go into one accumulator, smallest first, 64 of K long.
// bfloat16 operands sum 1024 of K.
//
// Roles (640 threads): warp 0 loads w, warp 2 loads b, warp 1 tensor memory
// and MMAs, warps 4 .. 11 epilogue (4 warps of 32 lanes for each 64 rows),
// warps 12 .. 19 split (F32).
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

constexpr int kTile = 128;               // of w's rows (logits) or columns (dx)
constexpr int kBK = 64;
constexpr int kUnit = kFewPiece;         // rows of w per unit of the logits' work
constexpr int kThreads = 640;
constexpr int kEpilogueWarp0 = 4;
constexpr int kEpilogueWarps = 8;
constexpr int kSplitWarp0 = 12;
constexpr int kSplitGroups = 2;          // take K blocks in turn
constexpr int kGroupWarps = 4;           // 32 lanes of tensor memory each
constexpr int kTmemCols = 512;
constexpr int kPartCols = 32;            // one part of a 128 x 64 tile in tensor memory
constexpr int kMostRings = 8;            // stages of b; of parts at most 4
constexpr int kSumBf16 = 16;             // K blocks per accumulator sum
constexpr int kSumStacked = 8;
constexpr int kStackedRows = 64;         // most rows with the parts of b stacked
constexpr int sum_blocks(bool f32, bool stacked) { return !f32 ? kSumBf16 : stacked ? kSumStacked : 1; }

template <bool F32>
struct Cfg {
  static constexpr int kWBytes = kTile * kBK * (F32 ? 4 : 2);
  static constexpr int kWStages = F32 ? 4 : 8;
  static constexpr int kParts = F32 ? 3 : 1;
  static constexpr int kBBytes = 96 * 1024;               // ring of b
  static constexpr int kSmem = 1024 + kWStages * kWBytes + kBBytes + 1024;
  static_assert(kBBytes >= 2 * kParts * kFewRows * kBK * 2, "two stages of b");
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

struct FewParams {
  int rows, n_pad;                       // T and the MMA's N
  int acc_cols, acc_bufs;                // columns of an accumulator (or three), buffers of it
  int b_stages, p_stages;                // stages of b, and of parts in tensor memory
  int width, vocab;
  int k_blocks;
  int units;                             // logits: of all classes
  FewClasses classes;
  int tiles, max_seg;                    // dx: ceil(width / 128), partials per tile
  long long sk_work;
  float* partials;                       // dx: [tile][max_seg][rows][128]
  float2* stats;
  long long ld_stats;
  void* exps;
  long long ld_exps;
  LossTargets targets;
  float* label_logit;
  unsigned* arrived;
  unsigned* err;
};

// Elements of the partial tiles, for the checked build.
[[maybe_unused]] __device__ __forceinline__ size_t partials_extent(const FewParams& p) {
  return static_cast<size_t>(p.tiles) * p.max_seg * p.rows * kTile;
}

// K blocks [k0, k1) of the tile of w that starts at row (or column) m0; for
// the logits row m0 of class cls, whose first `shift` columns are not its own.
struct Item {
  int m0, units, k0, k1, tile, seg;
  int cls, shift, unit;
};

// w as the kernel's maps read it.
template <int N>
struct WMaps {
  CUtensorMap of[N];
};

template <bool MN>
struct Items {
  long long x, end;

  __device__ __forceinline__ explicit Items(const FewParams& p) {
    const long long work = MN ? p.sk_work : p.units;
    x = sk_start(blockIdx.x, gridDim.x, work);
    end = sk_start(blockIdx.x + 1LL, gridDim.x, work);
  }
  __device__ __forceinline__ bool next(const FewParams& p, Item& w) {
    if (x >= end) return false;
    if (MN) {
      const long long ki = p.k_blocks;
      w.tile = static_cast<int>(x / ki);
      w.m0 = w.tile * kTile;
      w.units = kTile / kUnit;
      w.k0 = static_cast<int>(x - w.tile * ki);
      w.k1 = static_cast<int>(min(ki, w.k0 + (end - x)));
      w.seg = static_cast<int>(blockIdx.x) - sk_owner(w.tile * ki, gridDim.x, p.sk_work);
      w.cls = w.shift = w.unit = 0;
      x += w.k1 - w.k0;
    } else {   // within a class the least number of tiles, of about equal height
      constexpr int kMost = kTile / kUnit;
      w.unit = static_cast<int>(x);
      w.cls = w.unit / p.classes.units;
      const int in_class = w.unit - w.cls * p.classes.units;
      const int left = static_cast<int>(min(end - x, static_cast<long long>(p.classes.units - in_class)));
      const int tiles = (left + kMost - 1) / kMost;
      w.m0 = in_class * kUnit;
      w.units = (left + tiles - 1) / tiles;
      w.shift = (p.classes.shift0 + w.cls * p.classes.step) & p.classes.mask;
      w.k0 = 0;
      w.k1 = (p.width + w.shift + kBK - 1) / kBK;
      w.tile = w.seg = 0;
      x += w.units;
    }
    return true;
  }
};

// ---------------------------------------------------------------- primitives
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* desc, uint32_t bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(desc), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A in tensor memory: lane = row, each 32-bit column two consecutive K elements.
__device__ __forceinline__ void mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The order of floats as the order of signed integers (its own inverse).
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float unordered(int i) {
  return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF);
}

__device__ __forceinline__ float warp_max(float x) {
  return unordered(__reduce_max_sync(0xFFFFFFFFu, ordered(x)));
}

__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Sums over the warp of 16 values per lane by halving: after the step of
// lane bit b a lane keeps the half of the values that its bit selects.  Lane
// l ends with the sum of value (l >> 1), both lanes of a pair.
__device__ __forceinline__ float warp_sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {      // lane bits 16, 8, 4, 2
    const bool up = lane & (2 * n);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float give = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
      v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2 * n);
    }
  }
  return v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 1);
}

// Logits of one unit (a vocabulary entry v per lane) for 16 rows from t0 on,
// acc[at ..]: their statistics, powers and labels.  The 16 rows are
// independent, so that their reductions overlap.
template <bool F32>
__device__ __forceinline__ void logits_out(const FewParams& p, int piece, int v, int lane, int t0,
                                           const float (&acc)[64], int at) {
  const bool in = v < p.vocab;
  constexpr float kUp = F32 ? 0.0f : 15.0f;   // one part: powers times 2^15 (fp16)
  float top[16], e[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float z = in ? acc[at + j] : -INFINITY;
    top[j] = warp_max(z);
    e[j] = exp2_approx(fmaf(z - reference(top[j]), kLog2e, kUp));
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int t = t0 + j;
    if (t < p.rows && in && label_at(p.targets, t) == v) p.label_logit[t] = acc[at + j];
    if (t >= p.rows || p.exps == nullptr) continue;
    const size_t to = static_cast<size_t>(t) * p.ld_exps + v;
    if (!GEMM_IN_EXTENT(to, static_cast<size_t>(p.rows) * p.ld_exps, p.err, kSiteBoundsScratch))
      continue;
    if (F32)
      static_cast<float*>(p.exps)[to] = e[j];
    else
      static_cast<__half*>(p.exps)[to] = __float2half_rn(e[j]);
  }
  const float sum = warp_sum16(e, lane);
  float m = top[0];
#pragma unroll
  for (int j = 1; j < 16; ++j) m = lane >> 1 == j ? top[j] : m;
  const int t = t0 + (lane >> 1);
  const size_t stat = static_cast<size_t>(piece) * p.ld_stats + t;
  if ((lane & 1) == 0 && t < p.rows &&
      GEMM_IN_EXTENT(stat, static_cast<size_t>(p.units) * p.ld_stats, p.err, kSiteBoundsScratch))
    p.stats[stat] =
        make_float2(m, F32 ? sum : sum * (1.0f / 32768.0f));
}

// Bits of bfloat16 elements 2 i and 2 i + 1 that are not the first `shift`.
__device__ __forceinline__ uint32_t front_mask(int shift, int i) {
  return (2 * i >= shift ? 0xFFFFu : 0u) | (2 * i + 1 >= shift ? 0xFFFF0000u : 0u);
}

// ---------------------------------------------------------------- kernel
template <bool MN, bool F32, bool STACKED>
__global__ void __launch_bounds__(kThreads, 1)
    few_gemm_kernel(const __grid_constant__ WMaps<MN ? 1 : kFewMostClasses> tmW,
                    const __grid_constant__ CUtensorMap tmB, const FewParams p) {
  using C = Cfg<F32>;
  constexpr int SW = C::kWStages, PARTS = C::kParts;
  constexpr int SUM = sum_blocks(F32, STACKED);
  extern __shared__ uint8_t smem_dyn[];
  const uint32_t dyn0 = smem_addr(smem_dyn);
  const uint32_t base = (dyn0 + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_dyn + (base - dyn0);
  const uint32_t b_base = base + SW * C::kWBytes;
  const uint32_t bars = b_base + C::kBBytes;
  auto wfull = [&](int s) { return bars + 8u * s; };
  auto wempty = [&](int s) { return bars + 8u * (SW + s); };
  auto bfull = [&](int s) { return bars + 8u * (2 * SW + s); };
  auto bempty = [&](int s) { return bars + 8u * (2 * SW + kMostRings + s); };
  const uint32_t more_bars = bars + 8u * (2 * SW + 2 * kMostRings);
  auto pfull = [&](int s) { return more_bars + 8u * s; };          // parts in tensor memory
  auto pempty = [&](int s) { return more_bars + 8u * (4 + s); };
  auto accf = [&](int s) { return more_bars + 8u * (8 + s); };
  auto acce = [&](int s) { return more_bars + 8u * (10 + s); };
  const uint32_t drain_bar = more_bars + 8u * 12;
  const uint32_t tmem_slot = more_bars + 8u * 13;
  static_assert(8 * (2 * SW + 2 * kMostRings + 14) <= 1024, "barriers");

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);   // warp-uniform
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < SW; ++s) {
      mbar_init(wfull(s), 1);
      mbar_init(wempty(s), F32 ? kGroupWarps : 1);
    }
    for (int s = 0; s < kMostRings; ++s) {
      mbar_init(bfull(s), 1);
      mbar_init(bempty(s), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(pfull(s), kGroupWarps);
      mbar_init(pempty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(accf(s), 1);
      mbar_init(acce(s), kEpilogueWarps);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmW.of[0]);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = __shfl_sync(
      0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(base_ptr + (tmem_slot - base)), 0);
  const uint32_t parts0 = tmem_base + static_cast<uint32_t>(p.acc_bufs * p.acc_cols);
  grid_launch_dependents();
  grid_dependency_wait();   // global memory from here on
  if (!MN && blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0u;

  const uint32_t b_part_bytes = static_cast<uint32_t>(p.n_pad) * (kBK * 2);
  const uint32_t b_stage_bytes = PARTS * b_part_bytes;
  const int SB = p.b_stages;
  Item w;
  if (warp == 0) {
    // ------------------------------------------------------------ loads of w
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, armed = 0, last_ph = 0;
      bool ok = true;
      Items<MN> list(p);
      while (ok && list.next(p, w)) {
        for (int kb = w.k0; kb < w.k1; ++kb) {
          if (!mbar_wait(wempty(s), ph ^ 1u, p.err, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t st = base + s * C::kWBytes;
          const int k = kb * kBK;
          armed |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          if (MN) {
            mbar_arrive_expect_tx(wfull(s), C::kWBytes);
            constexpr int kCols = F32 ? 32 : 64;          // 128 bytes of a row
            constexpr uint32_t kBox = kBK * 128;
#pragma unroll
            for (int i = 0; i < kTile / kCols; ++i)
              tma_load_3d(st + i * kBox, &tmW.of[0], wfull(s), w.m0 + i * kCols, k, 0);
          } else {
            constexpr uint32_t kBox = kUnit * 128;
            const CUtensorMap* const map = &tmW.of[w.cls];
            mbar_arrive_expect_tx(wfull(s), static_cast<uint32_t>(w.units) * kBox * (F32 ? 2 : 1));
            for (int u = 0; u < w.units; ++u) {
              if (F32) {
                tma_load_3d(st + (2 * u) * kBox, map, wfull(s), k, w.m0 + u * kUnit, 0);
                tma_load_3d(st + (2 * u + 1) * kBox, map, wfull(s), k + 32, w.m0 + u * kUnit, 0);
              } else {
                tma_load_3d(st + u * kBox, map, wfull(s), k, w.m0 + u * kUnit, 0);
              }
            }
          }
          if (++s == SW) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      for (int q = 0; q < SW; ++q)
        if (armed & (1u << q)) mbar_wait(wfull(q), (last_ph >> q) & 1u, p.err, kSiteDrainTma);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ loads of b
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, armed = 0, last_ph = 0;
      bool ok = true;
      Items<MN> list(p);
      while (ok && list.next(p, w)) {
        for (int kb = w.k0; kb < w.k1; ++kb) {
          if (!mbar_wait(bempty(s), ph ^ 1u, p.err, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t st = b_base + static_cast<uint32_t>(s) * b_stage_bytes;
          armed |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          mbar_arrive_expect_tx(bfull(s), b_stage_bytes);
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
            tma_load_3d(st + part * b_part_bytes, &tmB, bfull(s), kb * kBK, 0, w.cls * PARTS + part);
          if (++s == SB) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      for (int q = 0; q < SB; ++q)
        if (armed & (1u << q)) mbar_wait(bfull(q), (last_ph >> q) & 1u, p.err, kSiteDrainTma);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // bfloat16 operands, fp32 accumulator, M = 128, N = n_pad; A in tensor
    // memory is K-major
    const uint32_t idesc_n = static_cast<uint32_t>(p.n_pad >> 3) << 17;
    const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((MN && !F32 ? 1u : 0u) << 15) |
                            ((kTile >> 4) << 24);
    const uint32_t idesc = idesc0 + idesc_n;
    const bool issuer = elect_lane();
    int sa = 0, sb = 0, buf = 0;         // sa: stage of w, or of its parts
    uint32_t pha = 0, phb = 0, acc_ph = 0;
    const int SA = F32 ? p.p_stages : SW;
    bool ok = true;
    Items<MN> list(p);
    while (ok && list.next(p, w)) {
      for (int kb = w.k0; kb < w.k1; ++kb) {
        const bool open = (kb - w.k0) % SUM == 0;
        const bool got = (!open || mbar_wait(acce(buf), acc_ph ^ 1u, p.err, kSiteMmaAccEmpty)) &&
                         mbar_wait(bfull(sb), phb, p.err, kSiteMmaReady) &&
                         mbar_wait(F32 ? pfull(sa) : wfull(sa), pha, p.err, kSiteMmaReady);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * p.acc_cols);
        const uint32_t bst = b_base + static_cast<uint32_t>(sb) * b_stage_bytes;
        const bool close = (kb - w.k0 + 1) % SUM == 0 || kb == w.k1 - 1;
        const uint32_t at = F32 ? parts0 + static_cast<uint32_t>(sa * 3 * kPartCols)
                                : base + sa * C::kWBytes;
        if (!MN && !F32 && kb == 0 && w.shift != 0) {
          // what lies in front of the rows (the first of eight 16-byte pieces,
          // swizzled) might be infinite or no number: x's zeros do not do
          for (int r = lane; r < w.units * kUnit; r += 32) {
            uint4* const front =
                reinterpret_cast<uint4*>(base_ptr + sa * C::kWBytes + r * 128 + ((r & 7) << 4));
            uint4 f = *front;
            f.x &= front_mask(w.shift, 0);
            f.y &= front_mask(w.shift, 1);
            f.z &= front_mask(w.shift, 2);
            f.w &= front_mask(w.shift, 3);
            *front = f;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        if (issuer) {
          uint32_t more = open ? 0u : 1u;
          if constexpr (STACKED) {
            // by hi, mid and lo of w: 3, 2 and 1 parts of b
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                mma_bf16_tmem_a(acc + static_cast<uint32_t>(part * p.n_pad),
                                at + static_cast<uint32_t>(part * kPartCols + kk * 8),
                                smem_desc(bst + kk * 32, 16, 1024, 2), idesc0 + (3 - part) * idesc_n, more);
                more = 1u;
              }
            mma_commit(pempty(sa));
          } else if constexpr (F32) {
            // (lo, hi), (hi, lo), (mid, mid), (mid, hi), (hi, mid), (hi, hi)
#pragma unroll
            for (int combo = 0; combo < 6; ++combo) {
              const int pa = (0x001102 >> (4 * combo)) & 3, pb = (0x010120 >> (4 * combo)) & 3;
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                mma_bf16_tmem_a(acc, at + static_cast<uint32_t>(pa * kPartCols + kk * 8),
                                smem_desc(bst + pb * b_part_bytes + kk * 32, 16, 1024, 2), idesc, more);
                more = 1u;
              }
            }
            mma_commit(pempty(sa));
          } else {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
              mma_bf16(acc, MN ? smem_desc(at + kk * 2048, 8192, 1024, 2) : smem_desc(at + kk * 32, 16, 1024, 2),
                       smem_desc(bst + kk * 32, 16, 1024, 2), idesc, more);
              more = 1u;
            }
            mma_commit(wempty(sa));
          }
          mma_commit(bempty(sb));
          if (close) mma_commit(accf(buf));
        }
        __syncwarp();
        if (++sa == SA) {
          sa = 0;
          pha ^= 1u;
        }
        if (++sb == SB) {
          sb = 0;
          phb ^= 1u;
        }
        if (close && ++buf == p.acc_bufs) {
          buf = 0;
          acc_ph ^= 1u;
        }
      }
    }
    if (issuer) {
      mma_commit(drain_bar);
      mbar_wait(drain_bar, 0, p.err, kSiteDrainMma);
    }
    __syncwarp();
  } else if (warp >= kEpilogueWarp0 && warp < kEpilogueWarp0 + kEpilogueWarps) {
    // ------------------------------------------------------------ epilogue
    // rows t of x or g: half of the n_pad for each four warps, in 16s
    const int q = warp & 3;
    const int split = (p.n_pad / 16 + 1) / 2 * 16;
    const int col0 = ((warp - kEpilogueWarp0) >> 2) * split;
    const int cols = min(split, p.n_pad - col0);
    const uint32_t t_mine =
        tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col0);
    int buf = 0;
    uint32_t acc_ph = 0;
    bool ok = true;
    Items<MN> list(p);
    while (ok && list.next(p, w)) {
      float acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
      for (int kb = w.k0; kb < w.k1; kb += SUM) {
        const bool got = mbar_wait(accf(buf), acc_ph, p.err, kSiteEpilogueFull);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          if (ch * 16 < cols) {
            const uint32_t at = t_mine + static_cast<uint32_t>(buf * p.acc_cols + ch * 16);
            uint32_t v[16];
            tmem_ld_16cols(at, v);
            if constexpr (STACKED) {   // the two smaller sums first
              uint32_t mid[16], low[16];
              tmem_ld_16cols(at + static_cast<uint32_t>(p.n_pad), mid);
              tmem_ld_16cols(at + static_cast<uint32_t>(2 * p.n_pad), low);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                acc[ch * 16 + j] += __uint_as_float(v[j]) + (__uint_as_float(mid[j]) + __uint_as_float(low[j]));
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[ch * 16 + j] += __uint_as_float(v[j]);
            }
          }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce(buf));
        if (++buf == p.acc_bufs) {
          buf = 0;
          acc_ph ^= 1u;
        }
      }
      if (!ok) break;
      if (MN) {
        float* const part = p.partials +
                            (static_cast<size_t>(w.tile) * p.max_seg + w.seg) * p.rows * kTile +
                            q * 32 + lane;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (j < cols && col0 + j < p.rows &&
              GEMM_IN_EXTENT(part + static_cast<size_t>(col0 + j) * kTile - p.partials, partials_extent(p),
                             p.err, kSiteBoundsWork))
            part[static_cast<size_t>(col0 + j) * kTile] = acc[j];
      } else if (q < w.units) {
        const int v = w.cls + p.classes.count * (w.m0 + q * kUnit + lane);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          if (ch * 16 < cols)
            logits_out<F32>(p, w.unit + q, v, lane, col0 + ch * 16, acc, ch * 16);
      }
    }
  } else if (F32 && warp >= kSplitWarp0) {
    // ------------------------------------------------------------ split of w
    const int q = warp & 3;                               // 32 lanes of tensor memory
    const int group = (warp - kSplitWarp0) / kGroupWarps;
    const uint32_t t_mine = parts0 + (static_cast<uint32_t>(q * 32) << 16);
    int s = 0, sp = 0, turn = 0;
    uint32_t ph = 0, php = 0;
    bool ok = true;
    Items<MN> list(p);
    while (ok && list.next(p, w)) {
      for (int kb = w.k0; kb < w.k1; ++kb) {
        if (turn == group) {
          const bool got = mbar_wait(wfull(s), ph, p.err, kSiteTransformFull) &&
                           mbar_wait(pempty(sp), php ^ 1u, p.err, kSiteTransformEmpty);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint8_t* const st = base_ptr + s * C::kWBytes;
#pragma unroll
          for (int half = 0; half < 2; ++half) {            // 32 of the 64 K elements
            float x[32];
            if (MN) {          // four boxes of 64 K rows of 32 columns: lane = column
              const float* const src = reinterpret_cast<const float*>(st + q * (kBK * 128)) + lane;
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = src[(half * 32 + k) * 32];
            } else {           // per unit of 32 rows two boxes of 32 K elements, swizzled: lane = row
              const uint8_t* const src = st + (2 * q + half) * (kUnit * 128) + lane * 128;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 f = *reinterpret_cast<const float4*>(src + ((c ^ (lane & 7)) << 4));
                x[4 * c] = f.x;
                x[4 * c + 1] = f.y;
                x[4 * c + 2] = f.z;
                x[4 * c + 3] = f.w;
              }
              if (half == 0 && kb == 0) {   // what lies in front of the row
#pragma unroll
                for (int k = 0; k < 3; ++k)
                  if (k < w.shift) x[k] = 0.0f;
              }
            }
            if (half == 1) {   // the tile is in registers
              __syncwarp();
              if (lane == 0) mbar_arrive(wempty(s));
            }
            // hi: truncated (never overflows); mid and lo: what is left, to nearest
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t a = __float_as_uint(x[2 * i]), b = __float_as_uint(x[2 * i + 1]);
              u[i] = __byte_perm(a, b, 0x7632);
              x[2 * i] -= __uint_as_float(a & 0xFFFF0000u);
              x[2 * i + 1] -= __uint_as_float(b & 0xFFFF0000u);
            }
            const uint32_t at = t_mine + static_cast<uint32_t>(sp * 3 * kPartCols + half * 16);
            tmem_st_16cols(at, u);
#pragma unroll
            for (int part = 1; part < 3; ++part) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&h);
                x[2 * i] -= __uint_as_float(u[i] << 16);
                x[2 * i + 1] -= __uint_as_float(u[i] & 0xFFFF0000u);
              }
              tmem_st_16cols(at + static_cast<uint32_t>(part * kPartCols), u);
            }
          }
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull(sp));
        }
        turn = (turn + 1) % kSplitGroups;
        if (++s == SW) {
          s = 0;
          ph ^= 1u;
        }
        if (++sp == p.p_stages) {
          sp = 0;
          php ^= 1u;
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// dx[t][d] = scale * the tile's partials added in order (of row t, or of rows
// t and rows + t, the two parts'); one thread per element, 128 columns of 2
// rows per CTA.
template <class T>
__global__ void __launch_bounds__(256)
    few_reduce_kernel(const FewParams p, int ctas, int rows, T* dx, long long lddx, const float* scale) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int tile = blockIdx.x, t = blockIdx.y * 2 + threadIdx.x / kTile, l = threadIdx.x % kTile;
  const int d = tile * kTile + l;
  if (t >= rows || d >= p.width) return;
  const long long ki = p.k_blocks;
  const int nseg = sk_owner((tile + 1) * ki - 1, ctas, p.sk_work) - sk_owner(tile * ki, ctas, p.sk_work) + 1;
  const size_t step = static_cast<size_t>(p.rows) * kTile;
  const float* src = p.partials + tile * p.max_seg * step + static_cast<size_t>(t) * kTile + l;
  const size_t second = static_cast<size_t>(p.rows - rows) * kTile;   // 0: one part
  float v = 0.0f, low = 0.0f;
  for (int s = 0; s < nseg; ++s)
    if (GEMM_IN_EXTENT(src + s * step + second - p.partials, partials_extent(p), p.err, kSiteBoundsWork)) {
      v += __ldcg(src + s * step);
      if (second) low += __ldcg(src + s * step + second);
    }
  v += low;
  const size_t at = static_cast<size_t>(t) * lddx + d;
  if (GEMM_IN_EXTENT(at, stored_extent(rows, p.width, lddx), p.err, kSiteBoundsRows))
    dx[at] = from_f32<T>(v * __ldg(scale));
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

int blocks_of(int n, int per) { return (n - 1) / per + 1; }

// The dx product's split of K over the CTAs.
int plan_dx(FewParams& p, int rows, int width, int vocab, int num_sms) {
  p.rows = rows;
  p.width = width;
  p.vocab = vocab;
  p.k_blocks = blocks_of(vocab, kBK);
  p.tiles = blocks_of(width, kTile);
  p.sk_work = static_cast<long long>(p.tiles) * p.k_blocks;
  const int ctas = static_cast<int>(std::min<long long>(num_sms, p.sk_work));
  p.max_seg = 1;
  for (int i = 0; i < p.tiles; ++i) {
    const long long k0 = static_cast<long long>(i) * p.k_blocks;
    p.max_seg = std::max(p.max_seg, sk_owner(k0 + p.k_blocks - 1, ctas, p.sk_work) -
                                        sk_owner(k0, ctas, p.sk_work) + 1);
  }
  return ctas;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, int size, const void* ptr, long long ld,
            int rows, int cols, int parts, long long plane, int box_cols, int box_rows,
            CUtensorMapSwizzle swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tma_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(ld) * size;
  const cuuint64_t strides[2] = {row_bytes,
                                 parts > 1 ? static_cast<cuuint64_t>(plane) * size : row_bytes * dims[1]};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  return enc(map, type, 3, const_cast<void*>(ptr), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of w: for the logits one per class, its rows from the boundary
// below row c on.  (That of row 0 lies up to 14 bytes before w, in a 16-byte
// block that also holds w's first element; its values are masked.)
bool encode_w(const FewGemm& g, bool mn, CUtensorMap* maps) {
  const CUtensorMapDataType type = g.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int size = g.f32 ? 4 : 2, box_cols = 128 / size;
  if (mn)
    return encode(maps, type, size, g.w, g.ldw, g.vocab, g.width, 1, 0, box_cols, kBK,
                  g.f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  const FewClasses& k = g.classes;
  for (int c = 0; c < k.count; ++c) {
    const int shift = (k.shift0 + c * k.step) & k.mask;
    const char* const first = static_cast<const char*>(g.w) + (c * g.ldw - shift) * size;
    if (!encode(maps + c, type, size, first, g.ldw * k.count, (g.vocab - c + k.count - 1) / k.count,
                g.width + shift, 1, 0, box_cols, kUnit, CU_TENSOR_MAP_SWIZZLE_128B))
      return false;
  }
  return true;
}

template <bool MN, bool F32, bool STACKED>
int launch_one(const FewGemm& g, const FewParams& p, const WMaps<MN ? 1 : kFewMostClasses>& mw,
               const CUtensorMap& mb, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};   // bit per device
  auto kern = few_gemm_kernel<MN, F32, STACKED>;
  const unsigned long long bit = 1ull << (g.device % kMaxDevices);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<F32>::kSmem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    configured.fetch_or(bit);
  }
  if (launch_dependent(kern, dim3(grid), dim3(kThreads), Cfg<F32>::kSmem, stream, mw, mb, p) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return GEMM_F32_ELAUNCH;
  }
  return GEMM_F32_OK;
}

template <bool MN>
int launch_type(const FewGemm& g, bool stacked, const FewParams& p, const CUtensorMap& mb, int grid,
                cudaStream_t stream) {
  WMaps<MN ? 1 : kFewMostClasses> mw = {};
  if (!encode_w(g, MN, mw.of)) return GEMM_F32_ELAUNCH;
  if (!g.f32) return launch_one<MN, false, false>(g, p, mw, mb, grid, stream);
  return stacked ? launch_one<MN, true, true>(g, p, mw, mb, grid, stream)
                 : launch_one<MN, true, false>(g, p, mw, mb, grid, stream);
}

}  // namespace

FewClasses few_classes(bool f32, const void* w, long long ldw, int vocab) {
  const int size = f32 ? 4 : 2;
  FewClasses c = {1, 0, 0, 0, 16 / size - 1};
  while (c.count * ldw * size % 16 != 0) c.count *= 2;
  c.units = blocks_of(blocks_of(vocab, c.count), kUnit);
  c.shift0 = static_cast<int>(reinterpret_cast<uintptr_t>(w) % 16) / size;
  c.step = static_cast<int>(ldw & c.mask);
  return c;
}

size_t few_gemm_scratch(int rows, int width, int vocab, int num_sms) {
  FewParams p = {};
  plan_dx(p, rows, width, vocab, num_sms);
  return sizeof(float) * p.tiles * p.max_seg * rows * kTile;
}

int launch_few_gemm(const FewGemm& g, cudaStream_t stream, int* launches) {
  if (g.rows < 1 || g.rows > kFewRows) return GEMM_F32_EINVAL;
  const bool dx = g.dx != nullptr;
  FewParams p = {};
  int grid;
  if (dx) {
    grid = plan_dx(p, g.rows, g.width, g.vocab, g.num_sms);
    p.partials = g.partials;
  } else {
    p.rows = g.rows;
    p.width = g.width;
    p.vocab = g.vocab;
    p.classes = g.classes;
    p.units = p.classes.count * p.classes.units;
    if (g.vocab < p.classes.count) return GEMM_F32_EINVAL;
    grid = std::min(p.units, g.num_sms);
    p.stats = g.stats;
    p.ld_stats = g.ld_stats;
    p.exps = g.exps;
    p.ld_exps = g.ld_exps;
    p.targets = g.targets;
    p.label_logit = g.label_logit;
    p.arrived = g.arrived;
  }
  p.n_pad = blocks_of(g.rows, 16) * 16;
  // tensor memory: accumulators, then stages of parts (at least two, and a
  // second accumulator where that leaves three)
  const bool stacked = g.f32 && p.n_pad <= kStackedRows;
  p.acc_cols = stacked ? 3 * p.n_pad : p.n_pad;
  p.acc_bufs = stacked && 2 * p.acc_cols + 9 * kPartCols > kTmemCols ? 1 : 2;
  p.p_stages = std::min(4, (kTmemCols - p.acc_bufs * p.acc_cols) / (3 * kPartCols));
  p.b_stages = std::min(kMostRings, Cfg<true>::kBBytes / ((g.f32 ? 3 : 1) * p.n_pad * kBK * 2));
  p.err = g.err;
  CUtensorMap mb;
  const int parts = g.f32 ? 3 : 1, copies = dx ? 1 : p.classes.count;
  const bool shifted = !dx && !p.classes.aligned();
  if (!encode(&mb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.b.ptr, g.b.ld, g.rows,
              dx ? g.vocab : shifted ? static_cast<int>(g.b.ld) : g.width, copies * parts, g.b.plane, kBK,
              p.n_pad, CU_TENSOR_MAP_SWIZZLE_128B))
    return GEMM_F32_ELAUNCH;
  const int rc = dx ? launch_type<true>(g, stacked, p, mb, grid, stream)
                    : launch_type<false>(g, stacked, p, mb, grid, stream);
  if (rc != GEMM_F32_OK) return rc;
  ++*launches;
  if (dx) {
    const int rows = g.two ? g.rows / 2 : g.rows;
    const dim3 blocks(p.tiles, (rows + 1) / 2);
    const cudaError_t err =
        g.f32 ? launch_dependent(few_reduce_kernel<float>, blocks, dim3(256), 0, stream, p, grid, rows,
                                 static_cast<float*>(g.dx), g.lddx, g.scale)
              : launch_dependent(few_reduce_kernel<__nv_bfloat16>, blocks, dim3(256), 0, stream, p, grid, rows,
                                 static_cast<__nv_bfloat16*>(g.dx), g.lddx, g.scale);
    if (err != cudaSuccess) {
      (void)cudaGetLastError();
      return GEMM_F32_ELAUNCH;
    }
    ++*launches;
  }
  return GEMM_F32_OK;
}

}  // namespace gemm_f32_impl
