// overlap.hpp against sets of bytes: random small matrices in a small address range.  Prints the
// number of pairs that overlapped and of those that did not; exits with 1 at the first difference.
#include <cstdio>
#include <cstdlib>
#include <set>

#include "overlap.hpp"

int main() {
  srand(1);
  auto pick = [](int lo, int hi) { return lo + rand() % (hi - lo + 1); };
  long yes = 0, no = 0;
  for (int n = 0; n < 400000; ++n) {
    gc::Area m[2];
    std::set<uintptr_t> bytes[2];
    const int shared = pick(1, 12);
    for (int k = 0; k < 2; ++k) {
      m[k].at = (uintptr_t)pick(0, 60);
      m[k].width = pick(0, 6);
      m[k].stride = m[k].width + pick(0, 8);
      if (n % 2 && shared >= m[k].width) m[k].stride = shared;      // often the same stride
      m[k].rows = pick(0, 7);
      if (m[k].at)
        for (int r = 0; r < m[k].rows; ++r)
          for (int c = 0; c < m[k].width; ++c) bytes[k].insert(m[k].at + r * m[k].stride + c);
    }
    bool want = false;
    for (uintptr_t b : bytes[0]) want = want || bytes[1].count(b);
    if (gc::overlap(m[0], m[1]) != want || gc::overlap(m[1], m[0]) != want) {
      for (auto& a : m) printf("at %lu width %ld stride %ld rows %ld\n", (unsigned long)a.at, (long)a.width, (long)a.stride, (long)a.rows);
      printf("want %d\n", (int)want);
      return 1;
    }
    (want ? yes : no) += 1;
  }
  printf("%ld %ld\n", yes, no);
  return 0;
}
