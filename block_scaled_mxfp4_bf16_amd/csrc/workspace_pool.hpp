// Registry of library-owned workspaces, one per (device, stream); `thread`
// tells streams apart that share one handle (0 otherwise).
//
// A buffer that has been handed out is never freed while the process runs:
// a HIP graph captured earlier keeps its address, and replaying the graph
// writes tickets and partial sums there.  When a call needs more than the
// current buffer holds, a larger one replaces it for later calls and the old
// one is retired -- kept allocated -- so earlier graphs stay valid.  Growth
// at least doubles the size, so the memory retired over a process's life is
// at most about the size of the live buffer.
//
// A call of more than one launch hands data from one to the next through its
// buffer, so it holds the buffer of its stream until the last is enqueued
// (hold): the launches of two threads' calls on one stream would otherwise
// mix, and the second launch of one would read what the first of the other
// wrote.
//
// Free of HIP types: the allocator is passed in (the library binds it to
// hipMalloc plus a zero-fill launch), so the bookkeeping can be exercised on
// the host alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <memory>
#include <mutex>
#include <vector>

namespace mxfp4 {

template <class Alloc>
class WorkspacePool {
 public:
  // Ownership of a held buffer; the mutex outlives the registry's entry.
  class Lock {
   public:
    Lock() = default;
    explicit Lock(std::shared_ptr<std::mutex> m) : mutex_(std::move(m)), lock_(*mutex_) {}

   private:
    std::shared_ptr<std::mutex> mutex_;  // destroyed after lock_
    std::unique_lock<std::mutex> lock_;
  };

  explicit WorkspacePool(Alloc alloc) : alloc_(alloc) {}

  // Buffer of at least `need` bytes (rounded up to 256) for (device,
  // stream); *out is null for need == 0.  Returns the allocator's status
  // (0 for success); on failure the registry is unchanged.
  int get(int device, void *stream, size_t need, void **out, uint64_t thread = 0) {
    std::shared_ptr<std::mutex> unused;
    return find(device, stream, thread, need, out, &unused);
  }

  // As get, and returns once no other caller holds a buffer of (device,
  // stream); *lock then keeps it from others until it is released.  Locks
  // nothing for need == 0.
  int hold(int device, void *stream, size_t need, void **out, Lock *lock, uint64_t thread = 0) {
    std::shared_ptr<std::mutex> busy;
    if (int st = find(device, stream, thread, need, out, &busy)) return st;
    // Growth by the holder waited for leaves *out retired, which serves as well.
    if (busy) *lock = Lock(std::move(busy));
    return 0;
  }

  // Bytes held, live and retired (for tests).
  size_t live_bytes() const {
    std::lock_guard<std::mutex> lk(mu_);
    size_t n = 0;
    for (const Entry &e : live_) n += e.bytes;
    return n;
  }
  size_t retired_bytes() const {
    std::lock_guard<std::mutex> lk(mu_);
    size_t n = 0;
    for (const Entry &e : retired_) n += e.bytes;
    return n;
  }
  size_t retired_count() const {
    std::lock_guard<std::mutex> lk(mu_);
    return retired_.size();
  }

 private:
  struct Entry {
    int device;
    void *stream;
    uint64_t thread;
    void *ptr;
    size_t bytes;
    std::shared_ptr<std::mutex> busy;  // held by the call that uses the buffer
  };

  int find(int device, void *stream, uint64_t thread, size_t need, void **out, std::shared_ptr<std::mutex> *busy) {
    *out = nullptr;
    if (need == 0) return 0;
    need = (need + 255) & ~(size_t)255;
    std::lock_guard<std::mutex> lk(mu_);
    for (Entry &e : live_) {
      if (e.device != device || e.stream != stream || e.thread != thread) continue;
      if (e.bytes < need) {
        size_t bytes = e.bytes * 2 > need ? e.bytes * 2 : need;
        retired_.reserve(retired_.size() + 1);  // what throws comes before the buffer
        void *p = nullptr;
        if (int st = alloc_(device, stream, bytes, &p)) return st;
        retired_.push_back(e);
        e.ptr = p;
        e.bytes = bytes;
      }
      *out = e.ptr;
      *busy = e.busy;
      return 0;
    }
    live_.reserve(live_.size() + 1);
    auto mutex = std::make_shared<std::mutex>();
    void *p = nullptr;
    if (int st = alloc_(device, stream, need, &p)) return st;
    live_.push_back(Entry{device, stream, thread, p, need, std::move(mutex)});
    *out = p;
    *busy = live_.back().busy;
    return 0;
  }

  Alloc alloc_;
  mutable std::mutex mu_;
  std::vector<Entry> live_;
  std::vector<Entry> retired_;  // still allocated: earlier graphs may use them
};

}  // namespace mxfp4
