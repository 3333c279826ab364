// Prints half_turns of each (frequency's bits, position) read from the standard input.
#include <cstdio>

#include "page_turn.cuh"

int main() {
  unsigned f;
  int p;
  while (std::scanf("%u %d", &f, &p) == 2)
    std::printf("%a\n", lbx::paged::half_turns(p, lbx::paged::turns_of(f)));
}
