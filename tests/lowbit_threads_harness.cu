// Host-only: two threads whose calls on one handle fail with different messages,
// read all the while by both. Prints the number of reads, and of those that were
// neither of the two messages.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>

#include "../codebook_decode_gb300/csrc/kv8_cache.cu"

int main() {
  qtts_kv8 c;
  c.cfg = {2, 8, 4, 128, 1e6f, 16, 4, 4096, 100};
  c.G = 152;
  const int32_t* i32 = (const int32_t*)0x1000;
  uint16_t* p = (uint16_t*)0x10000;
  const char* said[2] = {"qtts_kv8_append: layer 7 outside 0..1",
                         "qtts_kv8_append: k and v must be 8-byte aligned, with row strides that are multiples of 4 and hold a row"};
  std::atomic<long> reads{0}, torn{0};
  auto run = [&](int me) {
    for (int i = 0; i < 200000; ++i) {
      if (me == 0) qtts_kv8_append(&c, 7, 1, 1, 1, i32, i32, i32, 4, p, 512, p, 512, nullptr);
      else qtts_kv8_append(&c, 0, 1, 1, 1, i32, i32, i32, 4, p, 8, p, 512, nullptr);
      char seen[256];
      snprintf(seen, sizeof seen, "%s", qtts_kv8_last_error(&c));
      ++reads;
      if (strcmp(seen, said[0]) && strcmp(seen, said[1])) ++torn;
    }
  };
  std::thread a(run, 0), b(run, 1);
  a.join();
  b.join();
  printf("%ld %ld\n", reads.load(), torn.load());
  return 0;
}
