// The device memory that the library keeps from call to call, of one device
// (host code; Api is the CUDA runtime, or a stand-in in the tests).
//
// Each stream has a buffer of each kind, which its calls use in turn.  What
// orders their use is the stream, so nothing may be launched with a buffer
// that another call has grown meanwhile, and the kernels of two calls may not
// mix:
//   - A call holds its stream's entry from its first acquire() to its end
//     (WorkspaceCall, in every entry point that uses one): calls of several host
//     threads on one stream queue their kernels one call after the other.
//   - A graph keeps the addresses that its capture saw.  The scratch of a
//     captured call is therefore memory of the captured graph's own: it is
//     had during the capture and comes back once the graph and whatever was
//     instantiated from it are gone (a user object that the graph retains).
//     Replays run beside any other call.
//   - The products' buffers (split tail, operand copies) are the stream's own
//     in a capture too.  One that a capture has seen is never freed when the
//     stream's buffer grows, only by release().
// Nothing is allocated for the products during a capture: they do without.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <memory>
#include <mutex>
#include <unordered_map>
#include <vector>

namespace gemm_f32_impl {

// kSplitTail is zero when it is allocated; the others hold anything.
enum class Memory { kSplitTail, kPack, kScratch };

// The calling thread's call in progress, from its declaration on.
class WorkspaceCall {
 public:
  WorkspaceCall() : before_(current()) { current() = this; }
  ~WorkspaceCall() {
    if (held_) held_->unlock();
    current() = before_;
  }
  WorkspaceCall(const WorkspaceCall&) = delete;
  WorkspaceCall& operator=(const WorkspaceCall&) = delete;

 private:
  template <class Api>
  friend class Workspaces;
  static WorkspaceCall*& current() {
    static thread_local WorkspaceCall* call = nullptr;
    return call;
  }
  WorkspaceCall* const before_;
  const void* of_ = nullptr;               // the Workspaces and its entry that it uses
  void* entry_ = nullptr;
  std::mutex* held_ = nullptr;             // the entry's
};

template <class Api>
class Workspaces {
 public:
  using Stream = typename Api::Stream;
  using Graph = typename Api::Graph;

 private:
  struct Buffer {
    void* p = nullptr;
    size_t bytes = 0;
    bool captured = false;
  };
  struct GraphBuffer {
    void* p;
    size_t bytes;
    std::atomic<bool> held{true};          // by a graph; cleared on a thread of the runtime's
  };
  struct Entry {
    std::mutex mu;
    Stream stream;
    Buffer of[3];
    GraphBuffer* graph = nullptr;          // of the capture `capture`
    unsigned long long capture = 0;
  };

 public:
  // At least `bytes` of memory of a kind for the call in progress, which uses
  // one stream of one device; nullptr if they cannot be had.
  void* acquire(Stream stream, Memory kind, size_t bytes) {
    try {
      WorkspaceCall* const call = WorkspaceCall::current();
      if (!call) {                         // outside any: the memory is no one's once this returns
        const WorkspaceCall own;
        return acquire(stream, kind, bytes);
      }
      if (!call->held_) {
        Entry& e = entry(stream);
        e.mu.lock();                       // without entries_mu_, which release() holds while it waits for calls
        call->held_ = &e.mu;
        call->entry_ = &e;
        call->of_ = this;
      }
      if (call->of_ != this) return nullptr;
      Entry& e = *static_cast<Entry*>(call->entry_);
      if (e.stream != stream) return nullptr;
      unsigned long long id = 0;
      Graph graph = {};
      const bool capturing = Api::capturing(stream, &id, &graph);
      if (capturing && kind == Memory::kScratch) return of_graph(e, id, graph, bytes);
      Buffer& b = e.of[static_cast<int>(kind)];
      if (b.bytes < bytes && (capturing || !grow(b, kind, bytes))) return nullptr;
      if (capturing) b.captured = true;
      return b.p;
    } catch (...) {                        // the host's memory
      return nullptr;
    }
  }

  // Frees everything that no graph holds (what the products' captures saw
  // included), after the calls in progress.  The caller has synchronised the
  // device.
  void release() {
    std::lock_guard<std::mutex> all(entries_mu_);
    for (auto& e : entries_) {
      std::lock_guard<std::mutex> one(e.second->mu);
      for (Buffer& b : e.second->of) {
        if (b.p) Api::free(b.p);
        b = Buffer();
      }
    }
    std::lock_guard<std::mutex> kept(graphs_mu_);
    for (void* p : retired_) Api::free(p);
    retired_.clear();
    drop_graphs();
  }

 private:
  static size_t rounded(size_t bytes) {
    return (bytes + (size_t{1} << 20) - 1) & ~((size_t{1} << 20) - 1);
  }

  Entry& entry(Stream stream) {
    // the per-thread default stream is one handle for a stream of each thread
    static thread_local char thread;
    const void* const key = stream == Api::per_thread() ? static_cast<const void*>(&thread) : stream;
    std::lock_guard<std::mutex> lock(entries_mu_);
    std::unique_ptr<Entry>& e = entries_[key];
    if (!e) {
      e.reset(new Entry);
      e->stream = stream;
    }
    return *e;                             // never removed
  }

  bool grow(Buffer& b, Memory kind, size_t bytes) {
    {
      std::lock_guard<std::mutex> lock(graphs_mu_);
      if (b.p && b.captured) retired_.push_back(b.p);
      drop_graphs();
    }
    if (b.p && !b.captured) Api::free(b.p);   // synchronises the device: no kernel still uses it
    b = Buffer();
    const size_t want = rounded(bytes);
    void* const p = Api::alloc(want);
    if (!p) return false;
    if (kind == Memory::kSplitTail && !Api::zero(p, want)) {
      Api::free(p);
      return false;
    }
    b.p = p;
    b.bytes = want;
    return true;
  }

  // Memory of the graph that the stream is being captured into: one buffer for
  // the stream's calls of a capture, which the graph runs in turn.
  void* of_graph(Entry& e, unsigned long long id, Graph graph, size_t bytes) {
    if (e.graph && e.capture == id && e.graph->bytes >= bytes) return e.graph->p;
    std::lock_guard<std::mutex> lock(graphs_mu_);
    GraphBuffer* b = nullptr;
    for (auto& g : graphs_)                // the smallest that serves, of those that came back
      if (!g->held.load() && g->bytes >= bytes && (!b || g->bytes < b->bytes)) b = g.get();
    if (!b) {
      graphs_.reserve(graphs_.size() + 1);
      std::unique_ptr<GraphBuffer> made(new GraphBuffer);
      made->bytes = rounded(bytes);
      made->p = Api::alloc(made->bytes);
      if (!made->p) return nullptr;
      b = made.get();
      graphs_.push_back(std::move(made));
    }
    b->held.store(true);
    if (!Api::retain(graph, [](void* held) { static_cast<std::atomic<bool>*>(held)->store(false); }, &b->held)) {
      b->held.store(false);
      return nullptr;
    }
    e.graph = b;
    e.capture = id;
    return b->p;
  }

  void drop_graphs() {                     // under graphs_mu_, outside captures of the caller
    for (size_t i = 0; i < graphs_.size();) {
      if (graphs_[i]->held.load()) {
        ++i;
        continue;
      }
      Api::free(graphs_[i]->p);
      graphs_[i] = std::move(graphs_.back());
      graphs_.pop_back();
    }
  }

  std::mutex entries_mu_;
  std::unordered_map<const void*, std::unique_ptr<Entry>> entries_;
  std::mutex graphs_mu_;
  std::vector<std::unique_ptr<GraphBuffer>> graphs_;
  std::vector<void*> retired_;             // seen by captures of the products
};

}  // namespace gemm_f32_impl
