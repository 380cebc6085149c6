// What the C ABI's translation units (api.cpp, mx_api.cpp) share: the thread's error
// message and argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/nv4moe.h"

namespace nv4 {

// set the thread's error message and return `s`; ok() resets it
__attribute__((format(printf, 2, 3))) nv4_status fail(nv4_status s, const char *fmt, ...);
nv4_status ok();
nv4_status from_hip(hipError_t e, const char *what);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace nv4
