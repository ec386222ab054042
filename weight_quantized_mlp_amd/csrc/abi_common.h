// Argument and device checks shared by the C entry points (abi.cpp, abi_adapters.cpp).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/wqmlp.h"
#include "launch.h"

namespace wq {
namespace abi {

using wq::align256;

// hipError_t of the last WQ_ELAUNCH / WQ_EDEVICE on this host thread.
inline thread_local int g_last_hip = 0;

struct Rng {
  const void* p;
  size_t n;
};

inline bool overlaps(Rng a, Rng b) {
  if (a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline bool any_overlap(std::initializer_list<Rng> outs, std::initializer_list<Rng> ins) {
  for (const Rng& o : outs)
    for (const Rng& i : ins)
      if (overlaps(o, i)) return true;
  // outputs must not overlap each other either
  for (auto a = outs.begin(); a != outs.end(); ++a)
    for (auto b = a + 1; b != outs.end(); ++b)
      if (overlaps(*a, *b)) return true;
  return false;
}

inline bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (((uintptr_t)p & 15u) != 0) return false;
  return true;
}

inline bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return true;
  return false;
}

// ---- device checks (phase 2) ---------------------------------------------------------------------
constexpr int kMaxDev = 64;
inline std::once_flag g_arch_once[kMaxDev];
inline int g_arch_ok[kMaxDev];

inline int check_device(std::initializer_list<const void*> ptrs) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || dev < 0 || dev >= kMaxDev) {
    g_last_hip = (int)e;
    return WQ_EDEVICE;
  }
  std::call_once(g_arch_once[dev], [dev] {
    hipDeviceProp_t p;
    g_arch_ok[dev] = hipGetDeviceProperties(&p, dev) == hipSuccess && std::strncmp(p.gcnArchName, "gfx950", 6) == 0;
  });
  if (!g_arch_ok[dev]) return WQ_EARCH;
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    hipPointerAttribute_t a;
    e = hipPointerGetAttributes(&a, p);
    if (e != hipSuccess) {
      (void)hipGetLastError();  // clear the sticky error left by an unknown pointer
      g_last_hip = (int)e;
      return WQ_EDEVICE;
    }
    if (a.type != hipMemoryTypeDevice || a.device != dev) return WQ_EDEVICE;
  }
  return WQ_OK;
}

inline int launched(hipError_t e) {
  if (e != hipSuccess) {
    g_last_hip = (int)e;
    return WQ_ELAUNCH;
  }
  return WQ_OK;
}

constexpr int64_t kMaxDim = WQ_MAX_DIM;
// rows x columns of any activation or output matrix (keeps tile and grid counts in int)
constexpr int64_t kMaxElems = WQ_MAX_ELEMS;

inline size_t xsize(int dt) { return dt == WQ_F32 ? 4 : 2; }

inline size_t wbytes(int fmt, int64_t N, int64_t K) {
  return fmt == WQ_FMT_FP8W ? (size_t)N * (size_t)K : (size_t)N * (size_t)(K / 64) * 36;
}

}  // namespace abi
}  // namespace wq
