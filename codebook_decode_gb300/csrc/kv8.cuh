// kv8.cuh -- the 8-bit paged K/V cache: its layout in memory, the handle, and
// the device helpers that the append and attention kernels share.
//
// A block is one page (16 tokens) of one kv head's K or V: 16 * d codes and
// one fp32 scale. Codes are int8 values stored as code + 128 (an unsigned byte
// under a half's exponent is its value plus 1024, so widening to half needs
// no integer conversion; see widen()). K and V blocks of one (page, head) lie
// next to each other, so that one bulk copy brings both:
//   codes  [layer][page][kv head][K block 16 d | V block 16 d] bytes
//   scales [layer][page][kv head][K, V] fp32
// Inside a block the codes stand in the order in which the attention's MMA
// fragments take them, so that a lane's 16 bytes are one conflict-free load:
//   K: [d / 64][token 0..15][64 dims]
//   V: [d / 4][quad t 0..3][4 dims][tokens 2t, 2t + 1, 2t + 8, 2t + 9]
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "device_util.cuh"
#include "qtts_internal.h"

struct qtts_kv8 {
  qtts_kv8_config cfg{};
  int device = 0;
  int G = 0;  // SMs
  qtts::ErrorText err;
  uint8_t* codes = nullptr;
  float* scales = nullptr;
  float* rope_cos = nullptr;  // [max_context][d / 2], or nullptr: no rotation
  float* rope_sin = nullptr;
  int* dev_err = nullptr;
  std::vector<int32_t> free_ids;
  std::vector<uint8_t> page_used;
  std::vector<uint8_t> seen_now;  // qtts_kv8_free_pages's mark of ids seen in this call
};

namespace qtts {

constexpr int kKv8MaxBatch = 1024;
constexpr int kKv8MaxContext = 1 << 18;
constexpr int kKv8MaxGroup = 32;
// Scales below this are held as 0 (the block's values read back as 0): their
// reciprocals stay finite and their logarithms within the softmax's range.
constexpr float kKv8MinScale = 7.888609052210118e-31f;  // 2^-100

// What one layer's kernels need of the cache, and the sessions of a call.
struct Kv8View {
  uint8_t* codes;   // this layer's blocks
  float* scales;
  const float* rope_cos;
  const float* rope_sin;
  int nkv, pool_pages, max_context;
  int* err;
};
struct Kv8Batch {
  int B, n_rows, max_new;
  const int32_t* row_start;  // [B + 1], or nullptr: one row per session
  const int32_t* kv_len;     // [B]
  const int32_t* bt;         // [B][bt_stride]
  int bt_stride;
};
struct Kv8Session {
  int r0, n, L;  // first packed row, rows, tokens before them; n = 0: nothing to do
};

// The session's rows and length, checked: what does not fit its block table,
// the rotation table or the call's own limits sets the error word and is
// skipped. A negative kv_len marks an inactive session.
__host__ __device__ __forceinline__ Kv8Session kv8_session(const Kv8Batch& q, int b, int max_context, int* err) {
  Kv8Session s;
  s.r0 = q.row_start ? q.row_start[b] : b;
  const int r1 = q.row_start ? q.row_start[b + 1] : b + 1;
  s.L = q.kv_len[b];
  if (s.r0 < 0 || r1 < s.r0 || r1 > q.n_rows || r1 - s.r0 > q.max_new) {
    set_err(err, QTTS_DEV_BAD_SESSION);
    s.n = 0;
    return s;
  }
  s.n = r1 - s.r0;
  if (s.L < 0 || s.n == 0) {
    s.n = 0;
    return s;
  }
  const int cover = min((long long)max_context, (long long)q.bt_stride * kPage);
  if (s.n > cover || s.L > cover - s.n) {
    set_err(err, QTTS_DEV_BAD_SESSION);
    s.n = 0;
  }
  return s;
}

cudaError_t kv8_chunk_setup(int d);
bool kv8_chunk_fits(const Kv8View& v, const Kv8Batch& q, int group, long long pages);
size_t kv8_chunk_workspace(int d, int sms);
cudaError_t kv8_chunk(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                      int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, unsigned* arrived, float* part,
                      cudaStream_t s);
cudaError_t kv8_attention_setup(int d);
size_t kv8_attention_workspace(int d, int sms);
bool kv8_attention_fits(const Kv8View& v, const Kv8Batch& q, int group);
cudaError_t kv8_attention(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                          int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, void* work, cudaStream_t s);

}  // namespace qtts
