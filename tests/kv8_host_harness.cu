// Host-only checks of the 8-bit cache's and the 4-bit products' refusals: the
// translation units are compiled in, handles are filled in by hand, and every
// call here returns before it reaches the CUDA runtime. Prints one line per
// case: name, status, message. Also runs the per-session check (a device
// function that is plain arithmetic) on the CPU.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../codebook_decode_gb300/csrc/kv8_cache.cu"

static uint16_t* at(uintptr_t p) { return (uint16_t*)p; }

int main() {
  qtts_kv8 c;
  c.cfg = {2, 8, 4, 128, 1e6f, 16, 4, 4096, 100};
  c.G = 152;
  const int32_t* i32 = (const int32_t*)0x1000;
  uint16_t* ok = at(0x10000);
  const int W = 512, Q = 1024;  // row widths of k/v and q
  auto say = [&](const char* name, int rc) { printf("%s %d %s\n", name, rc, rc ? qtts_kv8_last_error(&c) : ""); };
  auto append = [&](const char* name, int layer, int B, int n, int mx, const int32_t* rs, const int32_t* kl, const int32_t* bt,
                    int bs, uint16_t* k, int64_t ks, uint16_t* v, int64_t vs) {
    say(name, qtts_kv8_append(&c, layer, B, n, mx, rs, kl, bt, bs, k, ks, v, vs, nullptr));
  };
  append("append_layer_low", -1, 1, 1, 1, i32, i32, i32, 4, ok, W, ok, W);
  append("append_layer_high", 2, 1, 1, 1, i32, i32, i32, 4, ok, W, ok, W);
  append("append_batch_0", 0, 0, 1, 1, i32, i32, i32, 4, ok, W, ok, W);
  append("append_batch_5", 0, 5, 5, 1, i32, i32, i32, 4, ok, W, ok, W);
  append("append_rows", 0, 1, -1, 1, i32, i32, i32, 4, ok, W, ok, W);
  append("append_max_new", 0, 1, 1, 0, i32, i32, i32, 4, ok, W, ok, W);
  append("append_stride", 0, 1, 1, 1, i32, i32, i32, 0, ok, W, ok, W);
  append("append_one_each_rows", 0, 2, 3, 1, nullptr, i32, i32, 4, ok, W, ok, W);
  append("append_one_each_max", 0, 2, 2, 2, nullptr, i32, i32, 4, ok, W, ok, W);
  append("append_null_len", 0, 1, 1, 1, i32, nullptr, i32, 4, ok, W, ok, W);
  append("append_null_table", 0, 1, 1, 1, i32, i32, nullptr, 4, ok, W, ok, W);
  append("append_null_k", 0, 1, 1, 1, i32, i32, i32, 4, nullptr, W, ok, W);
  append("append_null_v", 0, 1, 1, 1, i32, i32, i32, 4, ok, W, nullptr, W);
  append("append_k_align", 0, 1, 1, 1, i32, i32, i32, 4, at(0x10004), W, ok, W);
  append("append_k_narrow", 0, 1, 1, 1, i32, i32, i32, 4, ok, W - 4, ok, W);
  append("append_v_odd", 0, 1, 1, 1, i32, i32, i32, 4, ok, W, ok, W + 2);
  append("append_nothing", 0, 1, 0, 1, i32, i32, i32, 4, nullptr, 0, nullptr, 0);
  auto attend = [&](const char* name, uint16_t* q, int64_t qs, float scale, uint16_t* o, int64_t os, void* w) {
    say(name, qtts_kv8_attention(&c, 0, 1, 1, 1, i32, i32, i32, 4, q, qs, scale, o, os, w, nullptr));
  };
  attend("attend_null_q", nullptr, Q, 1.f, ok, Q, ok);
  attend("attend_null_out", ok, Q, 1.f, nullptr, Q, ok);
  attend("attend_q_narrow", ok, Q - 4, 1.f, ok, Q, ok);
  attend("attend_out_align", ok, Q, 1.f, at(0x10002), Q, ok);
  attend("attend_null_work", ok, Q, 1.f, ok, Q, nullptr);
  attend("attend_work_align", ok, Q, 1.f, ok, Q, at(0x10008));
  attend("attend_scale_nan", ok, Q, NAN, ok, Q, ok);
  attend("attend_scale_inf", ok, Q, INFINITY, ok, Q, ok);
  say("read_null_k", qtts_kv8_read(&c, 0, 1, 1, 1, i32, i32, i32, 4, nullptr, ok, nullptr));
  say("read_v_align", qtts_kv8_read(&c, 0, 1, 1, 1, i32, i32, i32, 4, ok, at(0x10004), nullptr));
  {
    qtts_kv8 big;
    big.cfg = {1, 1024, 1024, 128, 1e6f, 16, 1024, 262144, 100};
    const int rc = qtts_kv8_attention(&big, 0, 1024, 1024, 1, nullptr, i32, i32, 1 << 20, ok, 1024 * 128, 1.f, ok, 1024 * 128, ok, nullptr);
    printf("attend_too_much %d %s\n", rc, qtts_kv8_last_error(&big));
  }
  for (int i = 0; i < 10; ++i) {
    qtts_kv8_config f = {2, 8, 4, 128, 1e6f, 16, 4, 4096, 100};
    (i == 0 ? f.n_layers : i == 1 ? f.head_dim : i == 2 ? f.n_q_heads : i == 3 ? f.page_size : i == 4 ? f.max_batch
     : i == 5 ? f.max_context : i == 6 ? f.pool_pages : i == 7 ? f.n_kv_heads : f.n_layers) =
        i == 0 ? 0 : i == 1 ? 96 : i == 2 ? 6 : i == 3 ? 32 : i == 4 ? 1025 : i == 5 ? 262145 : i == 6 ? 0 : i == 7 ? 0 : 1;
    if (i == 8) f.rope_theta = -1.f;
    if (i == 9) f.n_q_heads = 4 * 33;
    qtts_kv8* out = &c;
    const int rc = qtts_kv8_create(&f, 0, &out);
    printf("config_%d %d %s\n", i, out ? -99 : rc, qtts_kv8_last_error(nullptr));
  }
  {
    qtts_kv8_config f = {1 << 26, 1, 1, 128, 1e6f, 16, 4, 4096, 1 << 26};
    qtts_kv8* out = &c;
    const int rc = qtts_kv8_create(&f, 0, &out);
    printf("config_bytes %d %s\n", out ? -99 : rc, qtts_kv8_last_error(nullptr));
  }
  say("free_not_allocated", (c.page_used.assign(100, 0), c.seen_now.assign(100, 0), [&] {
        const int32_t id = 3;
        return qtts_kv8_free_pages(&c, 1, &id);
      }()));
  say("free_twice", [&] {
    c.page_used[3] = 1;
    const int32_t ids[2] = {3, 3};
    return qtts_kv8_free_pages(&c, 2, ids);
  }());
  printf("still_used %d\n", (int)c.page_used[3]);
  say("alloc_too_many", [&] {
    int32_t ids[1];
    return qtts_kv8_alloc_pages(&c, 1, ids);
  }());
  printf("null_handle %d %d %d\n", qtts_kv8_append(nullptr, 0, 1, 1, 1, i32, i32, i32, 4, ok, W, ok, W, nullptr),
         qtts_kv8_status(nullptr, nullptr), qtts_kv8_free_count(nullptr));

  // the sessions' own check: rows r0, n, tokens before them, error word
  struct S {
    const char* name;
    int32_t rs[2], len;
    int n_rows, max_new, stride, max_context;
  } cases[] = {
      {"session_fits", {0, 3}, 61, 3, 3, 4, 4096},          {"session_past_table", {0, 4}, 61, 4, 4, 4, 4096},
      {"session_past_context", {0, 3}, 61, 3, 3, 40, 63},   {"session_inactive", {0, 1}, -1, 1, 1, 4, 4096},
      {"session_no_rows", {2, 2}, 10, 2, 1, 4, 4096},       {"session_rows_back", {2, 1}, 10, 2, 1, 4, 4096},
      {"session_rows_past", {0, 3}, 10, 2, 3, 4, 4096},     {"session_rows_many", {0, 3}, 10, 3, 2, 4, 4096},
      {"session_rows_negative", {-1, 1}, 10, 2, 2, 4, 4096}, {"session_huge", {0, 1}, 2147483647, 1, 1, 2147483647, 262144},
  };
  for (const S& s : cases) {
    int err = 0;
    const Kv8Batch q{1, s.n_rows, s.max_new, s.rs, &s.len, nullptr, s.stride};
    const Kv8Session r = kv8_session(q, 0, s.max_context, &err);
    printf("%s %d %d\n", s.name, r.n, err);
  }
  return 0;
}
