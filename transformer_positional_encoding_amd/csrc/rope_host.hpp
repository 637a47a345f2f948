// What the library's host code shares across its source files: the error of
// the calling thread and the current device's compute units.
#pragma once

#include <stdint.h>

#include <string>

#include "rope_partial.h"

namespace rope {

// The dispatch packet holds the grid size in work-items as a 32-bit number.
constexpr uint64_t kMaxGridItems = 0xFFFFFFFFull;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Keep `msg` as the calling thread's rope_last_error() and return st.
rope_status_t set_error(rope_status_t st, const std::string& msg);

// Compute units of the current device (cached per device).
rope_status_t device_cus(int* cus);

}  // namespace rope
