// Arithmetic of a group's slots cut into parts of `size`.  There may be 2^31 - 4,097 slots and parts of
// 2^30, whose signed sum would pass 2^31.  (Constant expressions, so that the host can run them too.)
#pragma once
#include <cstdint>

namespace tpc {

// parts of a run of `slots` (none where negative), `least` at least
constexpr int part_count(int slots, int size, int least) {
  const int c = slots > 0 ? (int)(((uint32_t)slots + (uint32_t)size - 1) / (uint32_t)size) : 0;
  return c > least ? c : least;
}
// end of the part that begins at `first`, of a run that ends at `hi`; both in [0, slots]
constexpr int part_end(int first, int hi, int size) { return hi - first > size ? first + size : hi; }

}  // namespace tpc
