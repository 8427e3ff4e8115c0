// Host-side state the entry points share: the thread's last error text and the
// optional per-pass event timing.
#pragma once
#include <hip/hip_runtime.h>

#include <string>
#include <utility>
#include <vector>

#include "../../include/dosa_indexer.h"

namespace dosa {

extern thread_local std::string g_err;

enum PassId { P_NORMS = 0, P_SCORE_SEED, P_SELECT_SEED, P_PLAN, P_BOUND, P_COMPACT, P_SURV_TILES, P_SURV_LISTS,
              P_SCORE_DENSE, P_SELECT_FINAL, P_PREP, P_PROBE, P_SEED_EXTRA, P_PROMPT, P_ATTEND, P_ATTEND_JOIN,
              P_APPEND, P_READ, P_WEIGHTS, P_WEIGHTS_JOIN, P_EVICT_SELECT, P_EVICT_MOVE, P_PAGES_ASSIGN,
              P_PAGES_RELEASE, P_PAGES_APPEND, P_PAGES_ATTEND, P_BLOCK_SELECT, P_BLOCK_ATTEND, P_COUNT };

struct Profiler {
  bool on = false;
  std::vector<hipEvent_t> pool;
  size_t used = 0;
  std::vector<std::pair<int, size_t>> recs;   // (pass, index of start event; stop = +1)
  hipEvent_t next() {
    if (used == pool.size()) {
      hipEvent_t e;
      if (hipEventCreate(&e) != hipSuccess) return nullptr;
      pool.push_back(e);
    }
    return pool[used++];
  }
};
extern thread_local Profiler g_prof;

struct PassScope {
  hipStream_t s;
  hipEvent_t stop = nullptr;
  PassScope(int pass, hipStream_t st) : s(st) {
    if (!g_prof.on) return;
    const size_t at = g_prof.used;
    hipEvent_t a = g_prof.next(), b = g_prof.next();
    if (!a || !b) return;
    (void)hipEventRecord(a, s);
    stop = b;
    g_prof.recs.push_back({pass, at});
  }
  ~PassScope() {
    if (stop) (void)hipEventRecord(stop, s);
  }
};

inline int fail_hip(hipError_t e, const char* what) {
  g_err = std::string(what) + ": " + hipGetErrorString(e);
  return DOSA_ERR_HIP;
}

inline int fail(int status, const std::string& text) {
  g_err = text;
  return status;
}

}  // namespace dosa
