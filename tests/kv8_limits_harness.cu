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
  auto fits = [](const char* name, int B, int n_rows, int max_new, int stride, int nkv, int group, int max_context) {
    Kv8View v{};
    v.nkv = nkv;
    v.max_context = max_context;
    const Kv8Batch q{B, n_rows, max_new, nullptr, nullptr, nullptr, stride};
    printf("%s %d\n", name, (int)kv8_attention_fits(v, q, group));
  };
  fits("fits_8_columns", 32, INT_MAX, 4, 128, 8, 2, 2048);
  fits("fits_16_columns", 32, INT_MAX, 8, 128, 8, 2, 2048);
  fits("fits_16_columns_one_session", 1, 1 << 30, 8, 16384, 8, 2, 262144);
  fits("fits_no_bounds", 1, INT_MAX, INT_MAX, 128, 8, 2, 2048);
  fits("fits_largest_prompt", 1, 262144, 262144, 16384, 8, 2, 262144);
  fits("fits_too_many_pages", 1024, 1024, 1, 16384, 1024, 1, 262144);
  fits("fits_too_many_rows", 1024, INT_MAX, INT_MAX, 16384, 8, 2, 262144);
  return 0;
}
