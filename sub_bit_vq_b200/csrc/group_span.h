// The sequences of a group, from device values that may be anything. Plain C++,
// so that a host test runs the code that the kernels run.
#pragma once

#ifdef __CUDACC__
#define LOOPVQ_HD __host__ __device__ __forceinline__
#else
#define LOOPVQ_HD inline
#endif

namespace loopvq {

// Sequences [lo, lo + n) of the group with the given start and end: the part
// inside [0, batch), at most max_group of them (none when the end is before the
// start). Both ends are clamped before they are subtracted, so that no difference
// leaves 32 bits.
struct GroupSpan {
  int lo, n;
};
LOOPVQ_HD GroupSpan group_span(int start, int end, int batch, int max_group) {
  GroupSpan s;
  s.lo = start < 0 ? 0 : start > batch ? batch : start;
  const int hi = end < 0 ? 0 : end > batch ? batch : end;
  s.n = hi < s.lo ? 0 : hi - s.lo;
  if (s.n > max_group) s.n = max_group;
  return s;
}

}  // namespace loopvq
