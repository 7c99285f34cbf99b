// What the C ABI's entry points (api.cpp, api_layers.cpp) share: checks of
// arguments and sizes.
#pragma once

#include <initializer_list>

#include "internal.hpp"

namespace sr {

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// n = a * b * c without overflow, all non-negative.
inline bool prod3(int64_t a, int64_t b, int64_t c, int64_t* n) {
  int64_t ab;
  return mul_ok(a, b, &ab) && mul_ok(ab, c, n);
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

inline sr_status check_workspace(void* ws, size_t have, size_t need) {
  if (need == 0) return SR_OK;
  if (ws == nullptr) return fail(SR_ERR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned(ws, kAlign)) return fail(SR_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(SR_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu needed", have, need);
  return SR_OK;
}

#define SR_REQUIRE(cond, ...)                                   \
  do {                                                          \
    if (!(cond)) return fail(SR_ERR_INVALID_ARGUMENT, __VA_ARGS__); \
  } while (0)

inline size_t elem_size(sr_dtype t) { return t == SR_BF16 ? 2 : 4; }

inline bool is_dtype(sr_dtype t) { return t == SR_F32 || t == SR_BF16; }

// Whether two ranges of bytes (of any length, none of them NULL) share memory.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a_bytes > 0 && b_bytes > 0 && x < y + uintptr_t(b_bytes) &&
         y < x + uintptr_t(a_bytes);
}

}  // namespace sr
