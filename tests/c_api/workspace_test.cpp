// csrc/workspace.h on a stand-in for the CUDA runtime: what is allocated,
// freed and held when, by streams, captures, graphs and host threads.
// Prints "ok <part>" for each part that passes.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <set>
#include <thread>
#include <vector>

#include "../../accelerator_row_major_gb300/csrc/workspace.h"

#define CHECK(c)                                               \
  do {                                                         \
    if (!(c)) {                                                \
      std::printf("line %d: %s\n", __LINE__, #c);              \
      std::exit(1);                                            \
    }                                                          \
  } while (0)

struct FakeGraph {
  std::vector<std::pair<void (*)(void*), void*>> held;
  ~FakeGraph() {
    for (auto& h : held) h.first(h.second);
  }
};

struct Fake {
  using Stream = char*;
  using Graph = FakeGraph*;
  static std::map<void*, size_t> live;     // allocations
  static std::map<Stream, std::pair<unsigned long long, FakeGraph*>> captures;
  static int allocs, zeros, fail_allocs, fail_zeros, fail_retains;

  static Stream per_thread() { return reinterpret_cast<Stream>(2); }
  static bool capturing(Stream s, unsigned long long* id, Graph* g) {
    auto at = captures.find(s);
    if (at == captures.end()) return false;
    *id = at->second.first;
    *g = at->second.second;
    return true;
  }
  static void* alloc(size_t n) {
    if (fail_allocs) return nullptr;
    ++allocs;
    void* p = std::malloc(64);             // what the runtime hands out may have been another's
    std::memset(p, 0xA5, 64);
    live[p] = n;
    return p;
  }
  static void free(void* p) {
    CHECK(live.erase(p) == 1);
    std::free(p);
  }
  static bool zero(void* p, size_t) {
    ++zeros;
    if (fail_zeros) return false;
    std::memset(p, 0, 64);
    return true;
  }
  static bool retain(Graph g, void (*done)(void*), void* arg) {
    if (fail_retains) return false;
    g->held.emplace_back(done, arg);
    return true;
  }
};
std::map<void*, size_t> Fake::live;
std::map<char*, std::pair<unsigned long long, FakeGraph*>> Fake::captures;
int Fake::allocs, Fake::zeros, Fake::fail_allocs, Fake::fail_zeros, Fake::fail_retains;

using gemm_f32_impl::Memory;
using gemm_f32_impl::WorkspaceCall;
using Pool = gemm_f32_impl::Workspaces<Fake>;
static char streams[8];
static char* const s0 = &streams[0];
static char* const s1 = &streams[1];
constexpr size_t kMiB = size_t{1} << 20;

static void* get(Pool& pool, char* stream, Memory kind, size_t bytes) {
  const WorkspaceCall call;
  return pool.acquire(stream, kind, bytes);
}

static void growth() {
  Pool pool;
  void* const a = get(pool, s0, Memory::kScratch, 100);
  CHECK(a && Fake::live.at(a) == kMiB);
  CHECK(get(pool, s0, Memory::kScratch, kMiB) == a);
  CHECK(get(pool, s1, Memory::kScratch, 1) != a && get(pool, s0, Memory::kPack, 1) != a);
  CHECK(Fake::live.size() == 3);
  void* const b = get(pool, s0, Memory::kScratch, kMiB + 1);
  CHECK(Fake::live.at(b) == 2 * kMiB && Fake::live.size() == 3);   // the old one went
  const int zeros = Fake::zeros;
  const char* z = static_cast<char*>(get(pool, s0, Memory::kSplitTail, 1));
  CHECK(Fake::zeros == zeros + 1 && z[0] == 0 && z[63] == 0);
  z = static_cast<char*>(get(pool, s0, Memory::kSplitTail, 2 * kMiB));   // again, whatever its address
  CHECK(Fake::zeros == zeros + 2 && z[0] == 0 && z[63] == 0);
  Fake::fail_allocs = 1;
  CHECK(!get(pool, s0, Memory::kScratch, 5 * kMiB));
  Fake::fail_allocs = 0;
  CHECK(get(pool, s0, Memory::kScratch, 5 * kMiB));
  Fake::fail_zeros = 1;
  const size_t before = Fake::live.size();
  CHECK(!get(pool, s1, Memory::kSplitTail, 1) && Fake::live.size() == before);
  Fake::fail_zeros = 0;
  pool.release();
  CHECK(Fake::live.empty());
  CHECK(get(pool, s0, Memory::kScratch, 1));
  pool.release();
  CHECK(Fake::live.empty());
  std::printf("ok growth\n");
}

static void graphs() {
  Pool pool;
  void* const eager = get(pool, s0, Memory::kScratch, kMiB);
  auto* first = new FakeGraph;
  Fake::captures[s0] = {11, first};
  void* const a = get(pool, s0, Memory::kScratch, kMiB);
  CHECK(a && a != eager);
  CHECK(get(pool, s0, Memory::kScratch, 10) == a);       // the capture's next call
  void* const more = get(pool, s0, Memory::kScratch, 3 * kMiB);
  CHECK(more != a && Fake::live.count(a));                // what it launched before keeps its own
  Fake::captures[s1] = {11, first};                       // a branch of the same capture
  void* const branch = get(pool, s1, Memory::kScratch, 1);
  CHECK(branch != a && branch != more);
  Fake::captures.clear();
  auto* second = new FakeGraph;
  Fake::captures[s0] = {12, second};
  void* const b = get(pool, s0, Memory::kScratch, 1);
  CHECK(b != a && b != more && b != branch);
  Fake::captures.clear();
  get(pool, s0, Memory::kScratch, 64 * kMiB);             // a larger call on the stream
  pool.release();
  for (void* p : {a, more, branch, b}) CHECK(Fake::live.count(p));   // replays still use them
  CHECK(Fake::live.size() == 4);
  delete first;
  auto* third = new FakeGraph;
  Fake::captures[s1] = {13, third};
  const int allocs = Fake::allocs;
  CHECK(get(pool, s1, Memory::kScratch, 2 * kMiB) == more && Fake::allocs == allocs);   // came back
  Fake::fail_retains = 1;
  CHECK(!get(pool, s1, Memory::kScratch, 100 * kMiB));
  Fake::fail_retains = 0;
  Fake::captures.clear();
  delete second;
  delete third;
  pool.release();
  CHECK(Fake::live.empty());
  std::printf("ok graphs\n");
}

static void products_in_captures() {
  Pool pool;
  FakeGraph graph;
  void* const a = get(pool, s0, Memory::kSplitTail, kMiB);
  Fake::captures[s0] = {21, &graph};
  const int allocs = Fake::allocs;
  CHECK(get(pool, s0, Memory::kSplitTail, kMiB) == a);
  CHECK(!get(pool, s0, Memory::kSplitTail, 2 * kMiB) && !get(pool, s0, Memory::kPack, 1));
  CHECK(Fake::allocs == allocs && graph.held.empty());
  Fake::captures.clear();
  void* const b = get(pool, s0, Memory::kSplitTail, 2 * kMiB);
  CHECK(b != a && Fake::live.count(a));                   // the graph has its address
  void* const c = get(pool, s0, Memory::kSplitTail, 4 * kMiB);
  CHECK(c && Fake::live.size() == 2);                     // b went: no graph has its
  pool.release();
  CHECK(Fake::live.empty());
  std::printf("ok products_in_captures\n");
}

static void threads() {
  Pool pool;
  using std::chrono::milliseconds;
  std::atomic<int> step{0};
  std::thread other, apart, releasing;
  {
    const WorkspaceCall call;
    CHECK(pool.acquire(s0, Memory::kScratch, 1));
    CHECK(pool.acquire(s0, Memory::kPack, 1));            // a second buffer of the same call
    CHECK(!pool.acquire(s1, Memory::kPack, 1));           // a call uses one stream
    other = std::thread([&] {
      const WorkspaceCall mine;
      CHECK(pool.acquire(s0, Memory::kScratch, 9 * kMiB));
      CHECK(step.load() == 1);
      step = 2;
    });
    apart = std::thread([&] { CHECK(get(pool, s1, Memory::kScratch, 1)); });
    apart.join();                                         // another stream does not wait
    std::this_thread::sleep_for(milliseconds(100));
    CHECK(step.load() == 0);
    step = 1;
  }
  other.join();
  CHECK(step.load() == 2);
  {
    const WorkspaceCall call;
    void* const p = pool.acquire(s0, Memory::kScratch, 1);
    releasing = std::thread([&] {
      pool.release();
      step = 3;
    });
    std::this_thread::sleep_for(milliseconds(100));
    CHECK(step.load() == 2 && Fake::live.count(p));       // held to the end of the call
    CHECK(pool.acquire(s0, Memory::kPack, 1));
  }
  releasing.join();
  CHECK(Fake::live.empty());
  // the per-thread default stream: a buffer of each thread's
  void *a = get(pool, Fake::per_thread(), Memory::kScratch, 1), *b = nullptr;
  std::thread([&] { b = get(pool, Fake::per_thread(), Memory::kScratch, 1); }).join();
  CHECK(a && b && a != b);
  pool.release();
  std::printf("ok threads\n");
}

int main() {
  growth();
  graphs();
  products_in_captures();
  threads();
  return 0;
}
