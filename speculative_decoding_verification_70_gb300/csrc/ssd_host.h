// ssd_host.h -- host-side helpers shared by the files that hold C-ABI entry
// points: the launch profiler, the NVTX call range and the argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>
#include <vector>

#ifndef SSD_NO_NVTX
#include <nvtx3/nvToolsExt.h>
#endif

#include "../../include/ssd.h"

namespace ssd {

// ---------------------------------------------------------------------------
// launch profiler
// ---------------------------------------------------------------------------
struct ProfRecord {
  int kernel;
  cudaEvent_t a, b;
};
struct Profiler {
  std::mutex mu;
  bool on = false;
  int cap = 0;
  std::vector<cudaEvent_t> pool;
  std::vector<ProfRecord> recs;
  std::vector<const char*> names;
  std::vector<int> counts;
  int kernel_id(const char* n) {
    for (size_t i = 0; i < names.size(); ++i)
      if (strcmp(names[i], n) == 0) return static_cast<int>(i);
    names.push_back(n);
    counts.push_back(0);
    return static_cast<int>(names.size() - 1);
  }
};
extern Profiler g_prof;  // ssd_api.cu

// Brackets one kernel launch when profiling is on.  A phase scope
// (launch = false) brackets several launches, possibly on other streams
// joined back by events, and adds no launch to the count.
struct ProfScope {
  cudaStream_t s = nullptr;
  int rec = -1;
  ProfScope() = default;
  ProfScope(const char* name, cudaStream_t st, bool launch = true) { begin(name, st, launch); }
  void begin(const char* name, cudaStream_t st, bool launch = true) {
    s = st;
    if (!g_prof.on) return;
    std::lock_guard<std::mutex> lk(g_prof.mu);
    int id = g_prof.kernel_id(name);
    if (launch) g_prof.counts[id] += 1;
    size_t used = g_prof.recs.size();
    if (static_cast<int>(used) >= g_prof.cap) return;
    ProfRecord r;
    r.kernel = id;
    r.a = g_prof.pool[2 * used];
    r.b = g_prof.pool[2 * used + 1];
    if (cudaEventRecord(r.a, s) != cudaSuccess) return;
    g_prof.recs.push_back(r);
    rec = static_cast<int>(used);
  }
  void end() {
    if (rec < 0) return;
    std::lock_guard<std::mutex> lk(g_prof.mu);
    cudaEventRecord(g_prof.recs[rec].b, s);
    rec = -1;
  }
  ~ProfScope() { end(); }
  ProfScope(const ProfScope&) = delete;
  ProfScope& operator=(const ProfScope&) = delete;
};

// One NVTX range per library call (header-only NVTX3: a no-op unless a
// profiler such as Nsight Systems or Nsight Compute injects itself).
struct CallRange {
#ifndef SSD_NO_NVTX
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
#else
  explicit CallRange(const char*) {}
#endif
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

inline cudaStream_t S(ssd_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline ssd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t esize(ssd_dtype dt) { return dt == SSD_BF16 ? 2 : 4; }

inline bool dtype_ok(ssd_dtype dt) { return dt == SSD_F32 || dt == SSD_BF16; }

// 16-byte vector loads are legal when every row start is 16-byte aligned.
inline bool vec_ok(const void* base, int64_t bstride, int V, ssd_dtype dt) {
  const size_t s = esize(dt);
  return aligned(base, 16) && (static_cast<size_t>(bstride) * s) % 16 == 0 &&
         (static_cast<size_t>(V) * s) % 16 == 0;
}

inline char* wsp(void* ws, size_t off) { return static_cast<char*>(ws) + off; }

}  // namespace ssd
