// How the norms at a block's ends lay their rows out: lanes, groups, chunks and
// the ring in shared memory, by rules on sizes and types.  Host code without a
// call of the CUDA runtime.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <numeric>

#include "block_norm.h"

namespace gemm_f32_impl {

namespace {

constexpr size_t kMostShared = 220 * 1024;   // dynamic; RowShared fits beside it
constexpr int kMostStages = 16;
constexpr size_t kLeastChunk = 16 * 1024;    // bytes of a stage, where there are rows enough

// What a thread has of a turn: elements of a row, rows.
struct Lane {
  int ne, rows;
};

// Lays out the rows of `in` over `ctas` CTAs, lanes, groups and ring; false
// where that cannot be.
bool plan_rows(RowPlan& plan, RowSource* in, int n, int vectors, int ctas, Lane lane, bool stats, int sums, bool aligned,
               int num_sms, size_t* bytes, int* grid) {
  const int ne = lane.ne;
  const int slice = ctas == 1 ? plan.width : ((plan.width - 1) / ctas / kSliceUnit + 1) * kSliceUnit;
  if (ctas > num_sms || slice > kRowWarps * 32 * ne) return false;
  plan.ctas = ctas;
  plan.slice = slice;
  plan.lanes = 32 * ((slice - 1) / (32 * ne) + 1);
  const long long units = num_sms / ctas;
  const size_t columns = static_cast<size_t>(vectors) * ne * plan.lanes * sizeof(float);
  // rows enough for all SMs; a thread's rows at a time only where there are so many
  plan.groups = static_cast<int>(std::min<long long>(kRowWarps * 32 / plan.lanes, (plan.rows - 1) / (units * lane.rows) + 1));
  if (lane.rows > 1 && plan.rows < units * lane.rows) return false;
  // copies of a forward turn that start at multiples of 32 KB all over the GPU meet on the same channels: 16 rows of
  // 1024 in bfloat16 101 us (65536 of them), 12 rows 89; 8 of 2048 101, 6 90
  const uint32_t turn_bytes = source_bytes(in[0].size, slice) * plan.groups;
  if (!stats && plan.groups >= 8 && turn_bytes % 32768 == 0) plan.groups -= plan.groups / 4;
  // the same of a gradient's turns of 16 elements a thread at 16 KB: 8 rows of 1024 in bfloat16 150 us (65536 of them),
  // 7 rows 130; 16 of 512 77 (as many of them), 15 74; with 8 elements a thread 181 against 190 for 8 rows of 512 in fp32
  if (stats && ne == 16 && plan.groups >= 8 && turn_bytes % 16384 == 0) --plan.groups;
  // a stage of `rows` rows
  const auto stage_of = [&](int rows) {
    size_t stage = 0;
    for (int i = 0; i < n; ++i) {
      if (!in[i].p) continue;
      const size_t row = source_bytes(in[i].size, slice);
      in[i].packed = ctas == 1 && in[i].ld == static_cast<long long>(row);
      in[i].pitch = static_cast<uint32_t>(in[i].packed ? row : (row + 15) / 16 * 16 + (aligned || in[i].size < 2 ? 0 : 16));
      in[i].at = static_cast<uint32_t>(stage);
      stage += (static_cast<size_t>(rows) * in[i].pitch + 15) / 16 * 16 + (in[i].packed && !aligned ? 16 : 0);
    }
    plan.stats_at = stats ? static_cast<uint32_t>(stage) : 0u;
    return stage + (stats ? rows * kStats * sizeof(float) : 0);
  };
  size_t stage = 0, stages = 0;
  for (;; --plan.groups) {               // two turns in flight, or fewer groups
    plan.turn = plan.groups * lane.rows;
    plan.chunk = lane.rows;
    for (int rows = 2 * lane.rows; rows <= plan.turn && stage_of(plan.chunk) < kLeastChunk; rows += lane.rows) {
      bool loose = false;
      for (int i = 0; i < n; ++i) loose = loose || (in[i].p && !in[i].packed);
      if (plan.turn % rows == 0 && rows <= (loose ? kMostLoose : kMostChunk)) plan.chunk = rows;
    }
    stage = stage_of(plan.chunk);
    stages = columns < kMostShared ? (kMostShared - columns) / (stage + 16) : 0;
    if (stages >= 2u * (plan.turn / plan.chunk) || plan.groups == 1) break;
  }
  if (stages < 2) return false;
  // a multiple of the chunks of a turn, and of as many producers as cost no more than a quarter of the stages
  const int step = plan.turn / plan.chunk;
  const int most = static_cast<int>(std::min<size_t>(stages, std::max(kMostStages, 2 * step)));
  for (plan.producers = kProducers; plan.producers >= 1; plan.producers /= 2) {
    const int unit = std::lcm(step, plan.producers);
    plan.stages = most / unit * unit;
    if (plan.stages >= 2 * step && (4 * plan.stages >= 3 * most || plan.producers == 1)) break;
  }
  plan.stage_bytes = static_cast<uint32_t>(stage);
  plan.ring_at = static_cast<uint32_t>(columns);
  // the groups' sums take the place of the ring
  const size_t rows_end = columns + static_cast<size_t>(plan.stages) * stage;
  const size_t sums_end = static_cast<size_t>(sums) * plan.groups * ne * plan.lanes * sizeof(float);
  plan.bars_at = static_cast<uint32_t>(std::max(rows_end, sums_end));
  *grid = static_cast<int>(std::min<long long>(units, (plan.rows - 1) / plan.turn + 1)) * ctas;
  *bytes = plan.bars_at + 16u * plan.stages;
  return true;
}

// A layout's price: what a turn takes its threads, by its rows.  A turn costs a
// warp some 250 instructions besides 16 for each of its elements (counted: 380
// of 8 elements), and more where CTAs exchange sums; a group that is alone
// waits for all of them, half as long for each of two rows.
constexpr int kTurnCost = 250, kExchangeCost = 300, kElementCost = 16;

long long price(const RowPlan& plan, Lane lane) {
  const long long turn = kTurnCost + (plan.ctas > 1 ? kExchangeCost : 0) + static_cast<long long>(kElementCost) * lane.ne * lane.rows;
  return turn * plan.ctas * (plan.groups == 1 ? (lane.rows == 1 ? 24 : 20) : 16) / plan.turn;
}

// Warpgroups of threads that compute, and the producer's.
int cta_threads(const RowPlan& plan) { return (plan.groups * plan.lanes + 127) / 128 * 128 + kProducerThreads; }

// A row layout that a call may take.
template <int N>
struct Layout {
  RowPlan plan;
  RowSource in[N];
  size_t bytes = 0;
  int grid = 0;
  Lane lane = {0, 0};                    // ne 0: there is none
};

// The cheapest layout.
template <int N, int K>
Layout<N> best_layout(const RowPlan& plan, const RowSource (&in)[N], const Lane (&lanes)[K], bool stats,
                      int sums, const BlockLaunch& l) {
  Layout<N> best = {};
  long long least = 0;
  for (int ctas = 1; ctas <= kMostCtas; ctas *= 2) {
    for (int i = 0; i < K; ++i) {
      Layout<N> c = {};
      c.plan = plan;
      std::copy(in, in + N, c.in);
      c.lane = lanes[i];
      if (!plan_rows(c.plan, c.in, N, l.vectors, ctas, lanes[i], stats, sums, l.aligned, l.num_sms, &c.bytes, &c.grid)) continue;
      const long long cost = price(c.plan, lanes[i]);
      if (best.lane.ne == 0 || cost < least) {
        best = c;
        least = cost;
      }
    }
    // more CTAs a row are for rows that leave a CTA no second group, where there are rows for one
    if (best.lane.ne && (best.plan.groups > 1 || plan.rows <= l.num_sms)) break;
  }
  return best;
}

// What a thread has of many rows, besides the 8 elements of one: two rows of
// them, or one row of 16, by the registers that the form's sums leave
// (8192 x 4096 bfloat16, with a gate per channel 83 us against 92 with one row
// of 8 and 119 with one of 16; rms norms on both ends 79 with 16, 104 with 8).
constexpr Lane grad_lane(bool layer, bool post, bool channel) {
  return channel || !post ? Lane{8, 2} : layer ? Lane{8, 1} : Lane{16, 1};
}

}  // namespace
}  // namespace gemm_f32_impl
