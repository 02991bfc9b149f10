// The handle behind the C ABI and what every entry point uses of it: device
// selection, error reporting, and counted, optionally timed launches.
#pragma once

#include <mutex>
#include <string>
#include <vector>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "muon.h"

struct muon_handle_s {
  // of everything below that a call reads or writes on the host (HandleLock)
  std::recursive_mutex mutex;
  int device = 0;
  int num_sms = 0;
  size_t ws_limit = size_t(16) << 30;
  unsigned long long timeout_ns = 4000000000ull;
  void* ws = nullptr;
  size_t ws_cap = 0;
  void* desc = nullptr;
  size_t desc_cap = 0;
  // pinned staging buffers of the descriptor arena, used in turn, each with
  // the event after which the device has read it
  static constexpr int kStages = 3;
  void* hstage[kStages] = {};
  const void* hstage_dev[kStages] = {};   // the same memory as the device addresses it
  size_t hstage_cap[kStages] = {};
  cudaEvent_t stage_ev[kStages] = {};
  bool stage_pending[kStages] = {};
  int stage_next = 0;
  unsigned* err = nullptr;
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  std::string last;
  // per-launch event timing (muon_handle_set_profiling)
  struct ProfRec {
    cudaEvent_t a, b;
    int cls;
    int tag;
  };
  bool profiling = false;
  int prof_tag = -1;            // group index of the launches being issued
  std::vector<ProfRec> prof;
  size_t prof_used = 0;
  uint64_t launches = 0;
  bool use_pair = true;         // CTA-pair GEMMs for large groups (MUON_TC_PAIR=0 disables)
  bool pair_update = true;      // UPDATE / FINAL on pairs too (MUON_TC_PAIR=sym: symmetric products only)
  int pair_min_m = 1024;        // ragged m from here on runs its symmetric products on pairs too (MUON_TC_PAIR_MIN_M)
  int max_pairs = 0;
  bool final_tma = true;        // FINAL into bf16 destinations through tensor maps (MUON_FINAL_TMA=0 disables)
  bool f32_tc = true;           // fp32 standard method on the tensor cores, three bf16 planes (MUON_F32_TC=0:
                                // CUDA cores)
  int f32_tc_max_m = 2048;      // ... for groups up to this m (MUON_F32_TC_MAX_M); the products' fp32
                                // accumulation error grows with K = m (with two accumulators per tile:
                                // 2048 x 8192 5.7e-5, 4096 x 4096 7.5e-5, 4096 x 14336 1.0e-4 against
                                // the 1e-4 bar)
  // standard bf16 method: the next unit's preparation on a side stream while
  // the current unit's products run (MUON_OVERLAP=1)
  bool overlap = false;
  cudaStream_t side = nullptr;
  std::vector<cudaEvent_t> ovl_ev;
  // standard bf16 method on small sets: every same-shape group's chain on a
  // stream of its own, so small launches of different groups share the SMs
  // (MUON_CONCURRENT: 0 off, 1 whenever the groups fit the workspace limit
  // together; default: also only for sets of at most kConcMaxElements)
  int concurrent = -1;
  std::vector<cudaStream_t> conc;
  std::vector<cudaEvent_t> conc_ev;
};

namespace muon {

// The set call is made on the right device too: a thread that has called no
// CUDA function yet (autograd's, say) has no context before it, and tensor
// maps are not encoded without one.
struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

// Host threads share a handle (the torch calls' default one): each entry point
// holds it for the length of its call.  Entry points call one another.
class HandleLock {
 public:
  explicit HandleLock(muon_handle_t h) noexcept {
    try {
      lock_ = std::unique_lock<std::recursive_mutex>(h->mutex);
    } catch (...) {          // the lock itself failed: as before there was one
    }
  }

 private:
  std::unique_lock<std::recursive_mutex> lock_;
};

inline muon_status_t fail(muon_handle_t h, muon_status_t st, const std::string& msg) {
  if (h != nullptr) h->last = msg;
  return st;
}

inline muon_status_t cuda_fail(muon_handle_t h, cudaError_t e, const char* what) {
  return fail(h, MUON_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

#define MUON_CUDA_TRY(expr, what)                  \
  do {                                             \
    cudaError_t e_ = (expr);                       \
    if (e_ != cudaSuccess) return cuda_fail(h, e_, what); \
  } while (0)

constexpr size_t kMaxProfRecords = size_t(1) << 20;

inline int prof_start(muon_handle_t h, int cls, cudaStream_t s) {
  if (!h->profiling || h->prof_used >= kMaxProfRecords) return -1;
  if (h->prof_used == h->prof.size()) {
    muon_handle_s::ProfRec r{};
    if (cudaEventCreate(&r.a) != cudaSuccess || cudaEventCreate(&r.b) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    h->prof.push_back(r);
  }
  const int slot = static_cast<int>(h->prof_used++);
  h->prof[slot].cls = cls;
  h->prof[slot].tag = h->prof_tag;
  cudaEventRecord(h->prof[slot].a, s);
  return slot;
}

inline void prof_stop(muon_handle_t h, int slot, cudaStream_t s) {
  if (slot >= 0) cudaEventRecord(h->prof[slot].b, s);
}

// Launch one kernel: optional event timing and the launch counter.
#define MUON_LAUNCH(cls, expr, what)                       \
  do {                                                     \
    const int slot_ = prof_start(h, (cls), stream);        \
    cudaError_t e_ = (expr);                               \
    if (e_ != cudaSuccess) return cuda_fail(h, e_, what);  \
    prof_stop(h, slot_, stream);                           \
    ++h->launches;                                         \
  } while (0)

}  // namespace muon
