// Host-side argument checks of the key-value cache, attention and log
// probability entry points (the same rules as those in gguf_qk.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/gguf_kv.h"
#include "kv_layout.hpp"

namespace gqk {

constexpr int kAbiDevices = 64;

// GGUF_QK_OK where the current device is a gfx950 (asked once per device).
inline int abi_device() {
  static std::atomic<int> seen[kAbiDevices];
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kAbiDevices) {
    (void)hipGetLastError();
    return GGUF_QK_ERR_DEVICE;
  }
  int c = seen[dev].load(std::memory_order_acquire);
  if (c == 0) {
    hipDeviceProp_t prop;
    const bool ok = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
                    std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    (void)hipGetLastError();
    c = ok ? 1 : -1;
    seen[dev].store(c, std::memory_order_release);
  }
  return c == 1 ? GGUF_QK_OK : GGUF_QK_ERR_DEVICE;
}

inline int abi_launched() { return hipGetLastError() == hipSuccess ? GGUF_QK_OK : GGUF_QK_ERR_LAUNCH; }

inline bool abi_aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline bool abi_overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && an > 0 && bn > 0 && a0 < b0 + (uintptr_t)bn && b0 < a0 + (uintptr_t)an;
}

// a * b, or -1 where it does not fit (a, b >= 0).
inline int64_t abi_mul(int64_t a, int64_t b) {
  int64_t r;
  return a < 0 || b < 0 || __builtin_mul_overflow(a, b, &r) ? -1 : r;
}

// Checks the cache description and fills the kernels' view of it.
int kv_view(const gguf_kv_cache* cache, KvView* view);

// The cache's bytes: K, V each, and weight, pos each.
inline int64_t kv_bytes(const KvView& c) { return c.n_pages * c.hkv * c.head_bytes; }
inline int64_t kv_plane_bytes(const KvView& c) { return c.n_pages * c.hkv * c.ps * 4; }

// Whether [p, p + n) touches any part of the cache.
inline bool kv_touches(const KvView& c, const void* p, int64_t n) {
  return abi_overlap(p, n, c.k, kv_bytes(c)) || abi_overlap(p, n, c.v, kv_bytes(c)) ||
         abi_overlap(p, n, c.weight, kv_plane_bytes(c)) || abi_overlap(p, n, c.pos, kv_plane_bytes(c));
}

}  // namespace gqk
