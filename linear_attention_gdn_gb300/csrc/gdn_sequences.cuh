// gdn_sequences.cuh -- what the recurrent steps share: the bounds of a sequence's tokens, and the strides of their rows.
#pragma once
#include <stdint.h>

namespace gdn {

// bounds of sequence n's tokens; false where they are none
__device__ __forceinline__ bool sequence_bounds(const int* cu, int n, int64_t T, int* t0, int* t1) {
  if (!cu) {
    *t0 = n;
    *t1 = n + 1;
    return true;
  }
  *t0 = cu[n];
  *t1 = cu[n + 1];
  return *t0 >= 0 && *t1 >= *t0 && *t1 <= T;
}

inline bool step_stride(int64_t* s, int heads, int esize) {
  if (*s == 0) *s = (int64_t)heads * 128;
  return *s >= (int64_t)heads * 128 && *s * esize % 16 == 0;
}

}  // namespace gdn
