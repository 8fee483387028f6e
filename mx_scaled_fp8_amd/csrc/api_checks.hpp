// Argument checks shared by the sources of the C ABI (not part of the ABI).
#pragma once

#include "common.hpp"

#define MX_CHECK(cond, ...)                                       \
  do {                                                            \
    if (!(cond)) return fail(MX_ERR_INVALID_ARG, __VA_ARGS__);    \
  } while (0)

// Validation done, dry-run honoured, device checked: the common preamble.
#define MX_PREAMBLE()                                   \
  do {                                                  \
    if (dry_run()) { clear_error(); return MX_OK; }     \
    const mx_status st_ = require_gfx950();             \
    if (st_ != MX_OK) return st_;                       \
  } while (0)
