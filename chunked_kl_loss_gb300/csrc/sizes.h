// Quotients and multiples rounded up.
#pragma once

#include <cstdint>

namespace fckl {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t rup(int64_t a, int64_t b) { return cdiv(a, b) * b; }

}  // namespace fckl
