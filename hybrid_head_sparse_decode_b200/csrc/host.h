// host.h -- host-side helpers shared by the library's entry points (internal):
// argument checks, device properties, the optional launch profiler.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cstdlib>
#include <mutex>
#include <vector>

#include "lychee.h"

namespace lychee {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether na bytes at a and nb bytes at b share any.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

inline lychee_status check_roles(const uint8_t* role, int Hq, int* n_sparse) {
  if (!role) return LYCHEE_ERR_INVALID_ARG;
  int ns = 0;
  for (int h = 0; h < Hq; ++h) {
    if (role[h] != LYCHEE_ROLE_SPARSE && role[h] != LYCHEE_ROLE_RETRIEVAL)
      return LYCHEE_ERR_INVALID_ARG;
    ns += role[h] == LYCHEE_ROLE_SPARSE;
  }
  if (n_sparse) *n_sparse = ns;
  return LYCHEE_OK;
}

// ---- tensor maps ----------------------------------------------------------------
// cuTensorMapEncodeTiled comes from the driver through the runtime's entry-point
// query, so the library needs no link against libcuda.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    cudaGetLastError();
  });
  return fn;
}

// ---- device properties -----------------------------------------------------------
inline int num_sms_current() {
  static std::mutex mu;
  static std::vector<int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  std::lock_guard<std::mutex> g(mu);
  if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    cache[dev] = n;
  }
  return cache[dev];
}

// ---- failure-path testing ---------------------------------------------------------
// For the attention kernels' bounded waits, read once from
// the environment: LYCHEE_TEST_WAIT_LIMIT_MS=<ms> shortens the limit after
// which their pipeline waits give up (`usual`: 2 s), and
// LYCHEE_TEST_WITHHOLD_ITEM=1 makes every CTA's builder withhold the
// announcement of its first work item (the 8-bit cache's kernel: makes every warp's
// first stage expect an arrival that never comes), so that the waits on it run out:
// the call then reports LYCHEE_ERR_TIMEOUT through lychee_check_device_error
// and every kernel returns.  Neither is meant for use outside tests.
inline uint64_t attn_wait_limit_ns(uint64_t usual) {
  static const uint64_t ns = [] {
    const char* v = std::getenv("LYCHEE_TEST_WAIT_LIMIT_MS");
    const long ms = v ? std::strtol(v, nullptr, 10) : 0;
    return ms > 0 ? (uint64_t)ms * 1000000ull : 0;
  }();
  return ns ? ns : usual;
}
inline bool attn_withhold_first_item() {
  static const bool on = [] {
    const char* v = std::getenv("LYCHEE_TEST_WITHHOLD_ITEM");
    return v && v[0] == '1';
  }();
  return on;
}

// ---- optional launch profiler ----------------------------------------------------
// Per-launch mode: two events around every launch.  Span mode: two events per
// stack call, before its first attention launch and after its last one, and
// none in between, so that the layers still overlap.
struct Profiler {
  std::mutex mu;
  bool on = false;
  bool spans = false;
  int cap = 0, n = 0;
  std::vector<cudaEvent_t> ev;
  std::vector<int32_t> kinds;
};
inline Profiler g_prof;

enum {
  kKindAttn = 0,
  kKindTopk = 1,
  kKindCombine = 2,
  kKindBuildBits = 3,
  kKindExport = 4,
  kKindTopkCombine = 5,
  kKindAttnSpan = 6,
  kKindAppend = 7
};

// Span mode: open (end = false) or close (end = true) the current stack call's
// attention span on `st`.
inline void span_mark(bool end, cudaStream_t st) {
  if (!g_prof.on || !g_prof.spans) return;
  std::lock_guard<std::mutex> g(g_prof.mu);
  if (!g_prof.on || !g_prof.spans) return;
  if (!end) {
    if (g_prof.n >= g_prof.cap) return;
    const int i = g_prof.n++;
    g_prof.kinds[i] = -1;   // open
    cudaEventRecord(g_prof.ev[2 * i], st);
  } else if (g_prof.n > 0 && g_prof.kinds[g_prof.n - 1] == -1) {
    const int i = g_prof.n - 1;
    g_prof.kinds[i] = kKindAttnSpan;
    cudaEventRecord(g_prof.ev[2 * i + 1], st);
  }
}

template <typename F>
cudaError_t timed(int kind, cudaStream_t st, F&& launch) {
  if (!g_prof.on || g_prof.spans) return launch();
  std::lock_guard<std::mutex> g(g_prof.mu);
  if (!g_prof.on || g_prof.spans || g_prof.n >= g_prof.cap) return launch();
  const int i = g_prof.n++;
  g_prof.kinds[i] = kind;
  cudaEventRecord(g_prof.ev[2 * i], st);
  const cudaError_t e = launch();
  cudaEventRecord(g_prof.ev[2 * i + 1], st);
  return e;
}

inline void fill_roles(uint32_t (&bits)[4], const uint8_t* role, int Hq) {
  bits[0] = bits[1] = bits[2] = bits[3] = 0;
  for (int h = 0; h < Hq; ++h)
    if (role[h] == LYCHEE_ROLE_RETRIEVAL) bits[h >> 5] |= 1u << (h & 31);
}

}  // namespace lychee
