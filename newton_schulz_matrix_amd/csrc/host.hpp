// host.hpp - what the C entry points share on the host: argument checks,
// workspace layout and type dispatch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nsortho.h"

namespace {

constexpr size_t kAlignTo = 256;
inline size_t align_up_to(size_t x) { return (x + kAlignTo - 1) / kAlignTo * kAlignTo; }
inline int64_t round_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline bool known(ns_dtype d) { return d == NS_BF16 || d == NS_FP16 || d == NS_FP32; }
inline int bytes_of(ns_dtype d) { return d == NS_FP32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline ns_status launched() { return hipGetLastError() == hipSuccess ? NS_OK : NS_ERR_HIP; }
// Grids of the kernels that loop over their rows stay below this many blocks
// (a launch may not have 2^32 threads).
constexpr int64_t kMaxBlocks = 1 << 20;

// Buffers carved out of a workspace in order.
struct Carver {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(int64_t count) {
    char* p = base ? base + used : nullptr;
    used += align_up_to((size_t)count * sizeof(T));
    return reinterpret_cast<T*>(p);
  }
};

inline bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % kAlignTo == 0);
}

// Calls f(IO{}, PT{}) for a data type and a parameter type that is the same
// or fp32.
template <class F>
ns_status with_types(ns_dtype io, ns_dtype pt, F&& f) {
  if (io == NS_FP32) return f(float{}, float{});
  if (io == NS_BF16) return pt == NS_FP32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
  return pt == NS_FP32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
}
template <class F>
ns_status with_type(ns_dtype io, F&& f) {
  if (io == NS_FP32) return f(float{});
  if (io == NS_BF16) return f(__bf16{});
  return f(_Float16{});
}

}  // namespace
