// Argument checks and error returns shared by the C ABI's source files.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../include/nvfp4ns.h"

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool dtype_ok(int d) { return d == NS_F32 || d == NS_BF16; }
inline size_t dtype_size(ns_dtype d) { return d == NS_F32 ? 4 : 2; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// Device arrays must be 16-byte aligned (the kernels move 16-byte vectors);
// single floats and words 4-byte aligned.
inline bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A byte range of device memory; null or empty ranges overlap nothing.
struct Span {
  const void* p;
  size_t n;
};
// Whether the written range `o` shares a byte with any of `others`.
inline bool hits(Span o, std::initializer_list<Span> others) {
  if (!o.p || o.n == 0) return false;
  for (const Span& t : others)
    if (t.p && t.n && overlaps(o.p, o.n, t.p, t.n)) return true;
  return false;
}

// A failed launch returns NS_ERR_HIP; with NVFP4NS_DEBUG set in the
// environment the HIP error and the failing call are also printed.
inline ns_status hip_failed(hipError_t e, const char* what, int line, const char* file = "api.hip") {
  if (std::getenv("NVFP4NS_DEBUG"))
    std::fprintf(stderr, "nvfp4ns: %s (%d) from %s, %s:%d\n", hipGetErrorString(e), (int)e, what,
                 file, line);
  return NS_ERR_HIP;
}

#define NS_TRY(call)                                          \
  do {                                                        \
    const hipError_t ns_e_ = (call);                          \
    if (ns_e_ != hipSuccess) return hip_failed(ns_e_, #call, __LINE__, __FILE_NAME__); \
  } while (0)

}  // namespace
