// Host-only: what the 8-bit cache's calls make of row counts and bounds of any
// size. The translation unit is compiled in; nothing reaches the CUDA runtime.
// Prints one line per case: name, value.
#include <climits>
#include <cstdio>

#include "../codebook_decode_gb300/csrc/kv8_cache.cu"

int main() {
  printf("pages_of_1 %d\n", touched_pages(1, 1, 4096));
  printf("pages_of_17 %d\n", touched_pages(17, 40, 4096));
  printf("pages_by_rows %d\n", touched_pages(1000, 18, 4096));
  printf("pages_by_context %d\n", touched_pages(1000, 1000, 33));
  printf("pages_no_bounds %d\n", touched_pages(INT_MAX, INT_MAX, kKv8MaxContext));
  printf("pages_near_the_end %d\n", touched_pages(INT_MAX - 20, INT_MAX, kKv8MaxContext));
  return 0;
}
