// Address ranges of a call's arguments, and small helpers of the host side.
// Plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hg.h"

namespace hg {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// An output may overlap nothing else.
struct Ranges {
  struct One {
    uintptr_t at;
    size_t bytes;
    bool written;
  };
  One r[HG_MAX_TP + 12];
  int n = 0;
  void add(const void *p, size_t bytes, bool written) {
    if (bytes) r[n++] = {reinterpret_cast<uintptr_t>(p), bytes, written};
  }
  bool clash() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((r[i].written || r[j].written) && r[i].at < r[j].at + r[j].bytes &&
            r[j].at < r[i].at + r[i].bytes)
          return true;
    return false;
  }
};

}  // namespace hg
