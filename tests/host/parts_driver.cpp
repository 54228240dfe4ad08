// Host-only driver for tests/test_host_parts.py: the arithmetic of groups cut into parts against the same in
// 64 bits, at the ends of what is declared.  Exits 0 when every check holds.
#include <algorithm>
#include <cstdio>

#include "parts.hpp"

int main() {
  const int64_t kSlots = 2147483647LL - 4096;
  int bad = 0;
  for (int64_t slots : {0LL, 1LL, 63LL, 64LL, 65LL, 100000LL, 1LL << 29, 1LL << 30, (1LL << 30) + 1, 3LL << 29, (long long)kSlots - 1,
                        (long long)kSlots})
    for (int64_t size : {1LL, 32LL, 64LL, 256LL, 5592448LL, 1LL << 29, (1LL << 30) - 64, 1LL << 30})
      for (int64_t least : {0, 1}) {
        const int64_t parts = std::max<int64_t>(least, (slots + size - 1) / size);
        bad += tpc::part_count((int)slots, (int)size, (int)least) != parts;
        bad += tpc::part_count((int)-slots, (int)size, (int)least) != least;
        // first, second, middle and last part of a run that ends at the last slot there may be
        const int64_t lo = kSlots - slots;
        for (int64_t t : {(int64_t)0, (int64_t)1, parts / 2, parts - 1}) {
          const int64_t first = std::min(lo + std::max<int64_t>(t, 0) * size, kSlots);
          bad += tpc::part_end((int)first, (int)kSlots, (int)size) != std::min(kSlots, first + size);
        }
      }
  std::printf("%d failures\n", bad);
  return bad != 0;
}
