// Integer helpers of the host code.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace bqm {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace bqm
