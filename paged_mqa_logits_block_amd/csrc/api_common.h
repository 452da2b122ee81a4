// What the files with the C-ABI entry points share: the calling thread's error
// message and the checks' small parts.
#pragma once

#include <stdint.h>

#include "qsaidx.h"

namespace qsa {

// records the message of a failed call and returns its status
__attribute__((format(printf, 2, 3))) qsa_status fail(qsa_status st, const char *fmt, ...);
// clears the message
qsa_status ok();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxBytes = (int64_t)1 << 62;

}  // namespace qsa
