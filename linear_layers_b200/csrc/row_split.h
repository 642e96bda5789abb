// row_split.h — how a row of logits is cut into 16-byte units, parts of blocks
// and groups of steps.  Launches and kernels call the same functions, so what a
// launch makes room for is what its blocks fill.  No CUDA header is needed.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TPL_HD __host__ __device__ __forceinline__
#else
#define TPL_HD inline
#endif

namespace tpl {

// A row of v elements from flat element f0 of a 16-byte-aligned matrix, kN
// elements to a unit: `head` elements up to the first 16-byte boundary, `units`
// whole units, `tail`.  Rows of any length are read in aligned units this way,
// and nothing outside the row is touched.  A row has the most units, v / kN,
// where head is 0.
template <int kN>
struct RowSplit {
  int head, units, tail;
  TPL_HD RowSplit(int64_t f0, int64_t v) {
    head = static_cast<int>((-f0) & (kN - 1));
    if (head > v) head = static_cast<int>(v);
    units = static_cast<int>((v - head) / kN);
    tail = static_cast<int>(v - head) - units * kN;
  }
};

// The units [first, last) of part `part` of `parts` equal ones; the last parts
// may have fewer or none.  No part has more units than part 0, nor than any
// part of a row with more of them.
struct Part {
  int first, last;
  TPL_HD Part(int units, int part, int parts) {
    const int per = (units + parts - 1) / parts;
    first = part * per < units ? part * per : units;
    last = first + per < units ? first + per : units;
  }
};

// Steps of `wide` units, and groups of 2^log steps.  A log that was taken for
// the widest part makes no more groups of a narrower one; a log taken anew for
// each part can: at most 32 groups are 17 for 33 steps, but 32 for 32.
TPL_HD int steps_of(int units, int wide) { return (units + wide - 1) / wide; }
TPL_HD int groups_of(int steps, int log) { return (steps + (1 << log) - 1) >> log; }
// the smallest log that makes at most `most` groups
TPL_HD int group_log_of(int steps, int most) {
  int log = 0;
  while (groups_of(steps, log) > most) ++log;
  return log;
}

}  // namespace tpl
