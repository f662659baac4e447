// Calls of more threads than a launch takes, host arithmetic.
//
// HIP takes less than 2^32 threads along a dimension of a grid, and does not
// always refuse more: a launch of 2^32 gave an error, one of 2^33 + 2^15 none,
// and left nearly all of its output unwritten. A call of more is launched in
// slices, one behind the other on its stream; its kernels add the slice's first
// workgroup to blockIdx.x.
#pragma once

#include <stdint.h>

namespace moe {

// Workgroups of a slice: whole runs of 16 tiles on each of 8 XCDs, so that
// tiles are dealt as in one launch.
inline int64_t slice_of(int threads) { return (((int64_t)1 << 32) - 1) / threads / 128 * 128; }

// launch(first, workgroups) for all `blocks` workgroups of `threads` threads
// (blocks up to 2^31 - 1), until one gives an error.
template <class F>
auto in_slices(int64_t blocks, int threads, F&& launch) -> decltype(launch(0u, 0u)) {
  const int64_t most = slice_of(threads);
  decltype(launch(0u, 0u)) e{};
  for (int64_t first = 0; first < blocks; first += most) {
    const int64_t left = blocks - first;
    e = launch((uint32_t)first, (uint32_t)(left < most ? left : most));
    if (e != decltype(e){}) break;
  }
  return e;
}

}  // namespace moe
