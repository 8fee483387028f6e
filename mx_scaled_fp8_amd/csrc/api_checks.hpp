// Argument checks shared by the sources of the C ABI (not part of the ABI).
#pragma once

#include "common.hpp"

#define MX_CHECK(cond, ...)                                       \
  do {                                                            \
    if (!(cond)) return fail(MX_ERR_INVALID_ARG, __VA_ARGS__);    \
  } while (0)

namespace mx {

// True if two tensors of so many bytes share none; a null pointer or no bytes share nothing.
inline bool apart(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !a || !b || a_bytes == 0 || b_bytes == 0 || x + a_bytes <= y || y + b_bytes <= x;
}

}  // namespace mx

// Validation done, dry-run honoured, device checked: the common preamble.
#define MX_PREAMBLE()                                   \
  do {                                                  \
    if (dry_run()) { clear_error(); return MX_OK; }     \
    const mx_status st_ = require_gfx950();             \
    if (st_ != MX_OK) return st_;                       \
  } while (0)
