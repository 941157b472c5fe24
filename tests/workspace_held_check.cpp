// Host-only check that a call keeps the library's workspace to itself from
// its first launch to its last (built by tests/test_workspace_held.py with
// g++: the two files of entry points, with the HIP calls and the launchers
// they make replaced by the stand-ins below; no GPU).
//
// A launcher that uses a workspace notes it as busy, gives way to other
// threads and clears the note; finding it busy means that the launches of two
// calls were mixed on one workspace.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <chrono>
#include <condition_variable>
#include <map>
#include <mutex>
#include <new>
#include <set>
#include <thread>
#include <vector>

#include "../block_scaled_mxfp4_bf16_amd/csrc/experts_internal.hpp"
#include "../block_scaled_mxfp4_bf16_amd/csrc/mxfp4_internal.hpp"

static std::mutex g_mu;
static std::set<void *> g_busy;
static std::map<std::thread::id, std::set<void *>> g_used;  // by each thread
static std::atomic<int> g_mixed{0}, g_calls{0};

// Two calls on different streams may be under way at once: with g_meet set,
// a launcher waits until a second one is inside.
static bool g_meet = false;
static int g_inside = 0;
static std::atomic<int> g_met{0};
static std::condition_variable g_cv;

static hipError_t two_launches(void *base) {
  ++g_calls;
  {
    std::unique_lock<std::mutex> lk(g_mu);
    if (!g_busy.insert(base).second) ++g_mixed;
    g_used[std::this_thread::get_id()].insert(base);
    if (g_meet) {
      ++g_inside;
      g_cv.notify_all();
      if (g_cv.wait_for(lk, std::chrono::seconds(10), [] { return g_inside >= 2; })) ++g_met;
    }
  }
  std::this_thread::sleep_for(std::chrono::microseconds(20));  // between the first launch and the second
  std::lock_guard<std::mutex> lk(g_mu);
  g_busy.erase(base);
  return hipSuccess;
}

// ---- host memory that runs out ----
static std::atomic<bool> g_no_memory{false};
static std::atomic<int> g_device_buffers{0};
void *operator new(size_t n) {
  void *p = g_no_memory ? nullptr : malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void *p) noexcept { free(p); }
void operator delete(void *p, size_t) noexcept { free(p); }

// ---- HIP ----
extern "C" {
hipError_t hipGetDevice(int *d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipMalloc(void **p, size_t n) {
  ++g_device_buffers;
  *p = aligned_alloc(256, (n + 255) & ~(size_t)255);
  return hipSuccess;
}
hipError_t hipFree(void *) { abort(); }  // a buffer in use would go
hipError_t hipGetSymbolAddress(void **, const void *) { abort(); }
const char *hipGetErrorName(hipError_t) { return "none"; }
}

// ---- launchers ----
namespace mxfp4 {
const size_t kBytes = 1 << 16;
int num_gemm_variants() { return 1; }
void gemm_variant_shape(int, Schedule *s) { *s = Schedule{4, 1, 1, 8, 4, 1, 0, 16, 1, 0, 0}; }
int find_gemm_variant(int, int, int, int, int, int, int, int, int) { return 0; }
size_t gemm_workspace_bytes(const Schedule &, int M, int, int) { return kTicketBytes + kBytes * (size_t)M; }
hipError_t launch_gemm(const Schedule &, const GemmArgs &a, bool, hipStream_t) { return two_launches(a.workspace); }
hipError_t launch_zero(void *, size_t, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize(const void *, int64_t, int64_t, void *, void *, bool, bool, hipStream_t) { abort(); }
hipError_t launch_preshuffle_b(const void *, const void *, int64_t, int64_t, void *, void *, hipStream_t) { abort(); }
hipError_t launch_prepare_b(const void *, int64_t, int64_t, void *, void *, bool, hipStream_t) { abort(); }
hipError_t launch_gemv(const GemvArgs &, hipStream_t) { abort(); }
hipError_t launch_combine(const CombineArgs &, hipStream_t) { abort(); }
size_t route_workspace_bytes(int64_t T, int64_t) { return kBytes * (size_t)T; }
hipError_t launch_route(const RouteArgs &a, hipStream_t) { return two_launches((char *)a.hist - kTicketBytes); }
size_t grouped_workspace_bytes(int64_t R, int64_t, int64_t) { return kBytes * (size_t)R; }
hipError_t launch_grouped(GroupedArgs a, hipStream_t) { return two_launches(a.ws - kTicketBytes); }
}  // namespace mxfp4

// ---- calls ----
static void *const P = (void *)0x100000;  // an aligned address, never read

static int call(int which, int size, void *stream) {
  switch (which & 3) {
    case 0:
      return mxfp4_gemm_grouped(P, 64, 8, P, P, 2, (int32_t *)P, nullptr, 1, P, 64, size, 64, 64, 0, nullptr, 0, stream);
    case 1:
      return mxfp4_moe_route(P, 0, 64, nullptr, size, 64, 2, 0, 1, (int32_t *)P, (float *)P, (int32_t *)P, (int32_t *)P,
                             (int32_t *)P, nullptr, 0, stream);
    case 2:
      return mxfp4_gemm(P, P, P, P, size, 64, 64, stream);
    default:
      return mxfp4_gemm_q(P, P, P, P, P, size, 64, 64, stream);
  }
}

static std::atomic<int> g_errors{0};

static void threads(int n, int calls, void *(*stream_of)(int)) {
  std::vector<std::thread> ts;
  for (int t = 0; t < n; ++t)
    ts.emplace_back([=] {
      for (int i = 0; i < calls; ++i)
        if (call(t + i, 1 + (i * 7 + t) % 5 * (i % 16 == 0 ? 4 : 1), stream_of(t)) != MXFP4_OK) ++g_errors;
    });
  for (auto &t : ts) t.join();
}

#define CHECK(c)                                                   \
  do {                                                             \
    if (!(c)) {                                                    \
      fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                    \
    }                                                              \
  } while (0)

int main(int argc, char **argv) {
  const char *what = argc > 1 ? argv[1] : "";
  if (!strcmp(what, "one_stream")) {
    threads(6, 150, [](int) -> void * { return (void *)0x40; });
    CHECK(g_errors.load() == 0 && g_calls.load() == 900);
    CHECK(g_mixed.load() == 0);
  } else if (!strcmp(what, "two_streams")) {
    g_meet = true;
    threads(2, 1, [](int t) -> void * { return (void *)(uintptr_t)(0x40 + 0x40 * t); });
    CHECK(g_errors.load() == 0 && g_met.load() == 2);
    CHECK(g_mixed.load() == 0);
  } else if (!strcmp(what, "stream_per_thread")) {
    // one handle for another stream in every thread: no buffer in common
    threads(4, 40, [](int) -> void * { return hipStreamPerThread; });
    CHECK(g_errors.load() == 0 && g_calls.load() == 160 && g_used.size() == 4);
    std::set<void *> all;
    size_t n = 0;
    for (auto &u : g_used) {
      n += u.second.size();
      all.insert(u.second.begin(), u.second.end());
    }
    CHECK(n == all.size());
    CHECK(mxfp4_reserve_bytes(1000, hipStreamPerThread) == MXFP4_OK);
  } else if (!strcmp(what, "no_host_memory")) {
    // a status, not an exception through the C entry; no device buffer that nothing remembers
    CHECK(call(2, 1, (void *)0x40) == MXFP4_OK);  // the schedule of this shape is remembered
    for (int which : {0, 1, 2}) {
      const int before = g_device_buffers;
      g_no_memory = true;
      const int st = call(which, 1, (void *)0x80);
      const int reserved = mxfp4_reserve_bytes(1000, (void *)0x80);
      g_no_memory = false;
      CHECK(st == MXFP4_ERR_HIP && reserved == MXFP4_ERR_HIP && g_device_buffers == before);
    }
    for (int which : {0, 1, 2}) CHECK(call(which, 1, (void *)0x80) == MXFP4_OK);
  } else {
    fprintf(stderr, "one_stream, two_streams, stream_per_thread or no_host_memory\n");
    return 2;
  }
  printf("%s ok\n", what);
  return 0;
}
