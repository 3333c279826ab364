// Prints turns_of of each number (a float's bits) read from the standard input.
#include <cstdio>

#include "page_turn.cuh"

int main() {
  unsigned f;
  while (std::scanf("%u", &f) == 1) std::printf("%llu\n", (unsigned long long)lbx::paged::turns_of(f));
}
