// Status reporting shared by the C entry points: the calling thread's last
// error text, and pointer-range checks.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/hclrmix.h"

namespace hc {

// Records the printf-style detail as the thread's last error and returns st.
hclrmix_status fail(hclrmix_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the thread's last error.
hclrmix_status ok();

struct Range {
  const char* name;
  uintptr_t lo, hi;
};

inline bool overlaps(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

}  // namespace hc
