// Host-side checks of device arrays that the operators around the expert layer
// share.  Internal header.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_q4.h"

namespace moeq4 {

inline bool args_aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
inline bool args_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}
// Bytes from the first element of a matrix to its last.
inline size_t args_span(long long rows, long long ld, long long cols, size_t es) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0;
}
// Bytes of an element of a MOE_Q4_DTYPE_*, 0 for another value.
inline size_t args_size(int dtype) {
  return dtype == MOE_Q4_DTYPE_F32 ? 4 : dtype == MOE_Q4_DTYPE_BF16 || dtype == MOE_Q4_DTYPE_F16 ? 2 : 0;
}

struct ArgSpan {
  const void* p;
  size_t n;
};
// Whether an output overlaps another output or an input (outs[i] may be given as NULL).
template <int NO, int NI>
bool args_alias(const ArgSpan (&outs)[NO], const ArgSpan (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (args_overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (args_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
  }
  return false;
}

}  // namespace moeq4
