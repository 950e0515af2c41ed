// csrc/block_plan.h on the host: every layout that it gives for the forms,
// types, widths, rows and strides below, checked; prints each ring as
// "ring groups rows chunk stages producers", a group's rows at a time second.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <tuple>

#include "../../accelerator_row_major_gb300/csrc/block_plan.h"

using namespace gemm_f32_impl;

#define CHECK(c)                                                                                              \
  do {                                                                                                        \
    if (!(c)) {                                                                                               \
      std::printf("line %d: %s (width %d, rows %lld, ctas %d, lanes %d, groups %d, chunk %d, stages %d)\n",   \
                  __LINE__, #c, p.width, p.rows, p.ctas, p.lanes, p.groups, p.chunk, p.stages);               \
      std::exit(1);                                                                                           \
    }                                                                                                         \
  } while (0)

static std::set<std::tuple<int, int, int, int, int>> rings;
static long layouts = 0;

template <int N>
void check(const RowPlan& p, const RowSource (&in)[N], Lane lane, int vectors, bool stats, int sums, bool aligned, int sms,
           size_t bytes, int grid) {
  ++layouts;
  // columns: each has a thread's element
  CHECK(p.lanes % 32 == 0 && p.lanes * lane.ne >= p.slice && static_cast<long long>(p.slice) * p.ctas >= p.width);
  CHECK(p.ctas == 1 || p.slice % kSliceUnit == 0);
  CHECK(p.groups >= 1 && p.groups * p.lanes <= 32 * kRowWarps && cta_threads(p) <= 32 * kRowWarps + kProducerThreads);
  CHECK(p.lanes == 32 || p.groups <= 8);                       // named barriers 1 .. 8, and 15
  // turns, chunks, stages
  CHECK(p.turn == p.groups * lane.rows && p.chunk % lane.rows == 0 && p.turn % p.chunk == 0);
  CHECK(lane.rows == 1 || p.rows >= static_cast<long long>(sms / p.ctas) * lane.rows);
  const int step = p.turn / p.chunk;
  CHECK(p.stages >= 2 * step && p.stages % step == 0 && p.stages % p.producers == 0);
  CHECK(p.producers == 1 || p.producers == 2 || p.producers == kProducers);
  rings.insert({p.groups, lane.rows, p.chunk, p.stages, p.producers});
  // shared memory: vectors, the ring, its barriers; the groups' sums from the first byte on, in front of the barriers
  const size_t slots = static_cast<size_t>(lane.ne) * p.lanes * sizeof(float);
  CHECK(p.ring_at == vectors * slots && p.ring_at % 16 == 0 && p.stage_bytes % 16 == 0 && p.bars_at % 16 == 0);
  CHECK(p.ring_at + static_cast<size_t>(p.stages) * p.stage_bytes <= p.bars_at);
  CHECK(sums * p.groups * slots <= p.bars_at);
  CHECK(bytes == p.bars_at + 16u * p.stages && bytes <= kMostShared && bytes + 5 * 1024 <= 227 * 1024);
  // a stage: each matrix's rows, statistics
  uint32_t at = 0;
  bool loose = false;
  for (int i = 0; i < N; ++i) {
    if (!in[i].p) continue;
    const uint32_t row = source_bytes(in[i].size, p.slice);
    const uint32_t above = aligned || in[i].size < 2 ? 0 : 15;       // a boundary
    const uint32_t last = (p.chunk - 1) * in[i].pitch + row;
    CHECK(in[i].at % 16 == 0 && in[i].at >= at);
    CHECK(in[i].packed ? in[i].pitch == row && p.ctas == 1 && in[i].ld == row : in[i].pitch % 16 == 0);
    at = in[i].at + (above + last + 15) / 16 * 16;
    loose = loose || !in[i].packed;
  }
  CHECK(!loose || p.chunk <= kMostLoose);
  CHECK(p.chunk <= kMostChunk);
  if (stats) {
    CHECK(p.stats_at > 0 && p.stats_at % 16 == 0 && at <= p.stats_at);
    at = p.stats_at + p.chunk * kStats * 4;
  }
  CHECK(at <= p.stage_bytes);
  CHECK(grid >= 1 && grid <= sms && grid % p.ctas == 0);
}

// Every layout of a call; returns whether there is one.
template <int N, int K>
bool layouts_of(const RowPlan& plan, const RowSource (&in)[N], const Lane (&lanes)[K], int vectors, bool stats, int sums,
                bool aligned, int sms) {
  bool some = false;
  for (int ctas = 1; ctas <= kMostCtas; ctas *= 2) {
    for (const Lane& lane : lanes) {
      RowPlan p = plan;
      RowSource m[N];
      std::copy(in, in + N, m);
      size_t bytes = 0;
      int grid = 0;
      if (!plan_rows(p, m, N, vectors, ctas, lane, stats, sums, aligned, sms, &bytes, &grid)) continue;
      some = true;
      check(p, m, lane, vectors, stats, sums, aligned, sms, bytes, grid);
    }
  }
  const BlockLaunch l = {vectors, aligned, true, 0, sms, nullptr, nullptr, nullptr};
  const Layout<N> best = best_layout(plan, in, lanes, stats, sums, l);
  const RowPlan& p = best.plan;
  CHECK((best.lane.ne != 0) == some);
  if (some) check(best.plan, best.in, best.lane, vectors, stats, sums, aligned, sms, best.bytes, best.grid);
  return some;
}

RowSource rows_of(int size, int width, bool packed) {
  RowSource m = {};
  m.p = reinterpret_cast<const char*>(4096);
  m.size = size;
  const long long row = source_bytes(size, width);
  if (size >= 2)
    m.ld = row + (packed ? 0 : 16);
  else                                                         // 8-bit rows: multiples of 16 bytes
    m.ld = (size ? (width + 31LL) / 32 * 32 : (row + 15) / 16 * 16) + (packed ? 0 : 16);
  return m;
}

int main() {
  const int widths[] = {1,    2,    7,    8,    31,   32,   33,   64,   74,   100,   128,   255,   256,   257,   500,  777,
                        1000, 1024, 1280, 2048, 2056, 4095, 4096, 4097, 5000, 8192,  8193,  12288, 16384, 16385, 20001, 32768,
                        32769, 40000, 65536, 131072};
  const long long many[] = {1, 3, 37, 151, 153, 305, 700, 1217, 2500, 5000, 100000, 1LL << 40};
  for (const int sms : {148, 152}) {
    for (const int width : widths) {
      for (const long long rows : many) {
        for (const int es : {2, 4}) {
          for (const bool packed : {false, true}) {
            for (const bool aligned : {false, true}) {
              if (aligned && width * es % 16) continue;
              RowPlan plan = {};
              plan.width = width;
              plan.rows = rows;
              for (int gate = kNoGate; gate <= kElementGate; ++gate) {
                for (int vectors = 1; vectors <= 5; ++vectors) {
                  RowSource in[kInputs] = {rows_of(es, width, packed), rows_of(es, width, packed)};
                  if (gate == kElementGate) in[kInGate] = rows_of(es, width, packed);
                  const Lane lanes[3] = {{8, 1}, {16, 1}, {32, 1}};
                  const bool some = layouts_of(plan, in, lanes, vectors, false, 0, aligned, sms);
                  const RowPlan& p = plan;
                  CHECK(some || width > 32768);
                }
                for (int form = 0; form < 16; ++form) {
                  const bool layer = form & 1, post = form & 2, saved = form & 4, dh = form & 8;
                  const bool by_channel = gate == kChannelGate || (layer && post && gate == kNoGate);
                  const bool branch = post || gate != kNoGate;
                  RowSource in[kGradInputs] = {};
                  in[kGradDy] = rows_of(es, width, packed);
                  if (dh) in[kGradDh] = rows_of(es, width, packed);
                  in[kGradH] = rows_of(saved ? 1 : es, width, packed);
                  if (saved) in[kGradHExponents] = rows_of(0, width, packed);
                  if (branch) in[kGradBranch] = rows_of(saved ? 1 : es, width, packed);
                  if (branch && saved) in[kGradBranchExponents] = rows_of(0, width, packed);
                  if (gate == kElementGate) in[kGradGate] = rows_of(es, width, packed);
                  const int vectors = post && by_channel ? 2 : 1 + post + (post && layer && gate != kNoGate) + (gate == kChannelGate);
                  const int most = (layer ? 2 : 1) + (post ? (layer ? 2 : 1) : 0) + (gate == kChannelGate);
                  const Lane lanes[2] = {{8, 1}, grad_lane(layer, post, by_channel)};
                  for (const int sums : {0, most}) {
                    const bool some = layouts_of(plan, in, lanes, vectors, true, sums, aligned, sms);
                    const RowPlan& p = plan;
                    CHECK(some || width > 32768);
                  }
                }
              }
            }
          }
        }
      }
    }
  }
  for (const auto& r : rings)
    std::printf("ring %d %d %d %d %d\n", std::get<0>(r), std::get<1>(r), std::get<2>(r), std::get<3>(r), std::get<4>(r));
  std::printf("ok %ld layouts\n", layouts);
  return 0;
}
