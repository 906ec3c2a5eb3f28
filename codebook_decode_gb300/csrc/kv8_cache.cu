// kv8_cache.cu -- the 8-bit paged K/V cache's handle, its append (position
// rotation and quantisation on the way in) and its read-back.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "kv8.cuh"

namespace qtts {
namespace {

// One warp per (page, head, K or V) block; a CTA takes up to 16 blocks of one
// page of one session.
constexpr int kMaxWarps = 16;

// The rotation table: angles in double (a position of a long context times a
// frequency loses its fraction in fp32), stored fp32.
__global__ void rope_table_kernel(float* cs, float* sn, int max_context, int half, double theta) {
  grid_dependency_wait();
  const int i = threadIdx.x;
  const double f = pow(theta, -(double)i / half);
  for (int p = blockIdx.x; p < max_context; p += gridDim.x) {
    double s, c;
    sincos((double)p * f, &s, &c);
    cs[(size_t)p * half + i] = (float)c;
    sn[(size_t)p * half + i] = (float)s;
  }
}

// Four bf16 as two pairs of fp32.
__device__ __forceinline__ void bf4(uint2 v, uint64_t& a, uint64_t& b) {
  a = pack2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
  b = pack2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
// largest magnitude of the three, NaN if one is
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_abs(float m, uint64_t a) {
  const float2 f = unpack2(a);
  return max_abs(m, f.x, f.y);
}
// Rounding to an integer by adding 1.5 * 2^23 (half-even, like the product
// before it in binary32); with 128 on top the low byte is the stored code. No
// clamp: x * inv is at most 127 (1 + 2^-22).
// The products stay scalar: the paired multiply and add were fused into one rounding.
__device__ __forceinline__ uint64_t code_bits(uint64_t x, float inv) {
  const float2 f = unpack2(x);
  return add2(pack2(__fmul_rn(f.x, inv), __fmul_rn(f.y, inv)), pack2(12583040.f, 12583040.f));
}
// the low bytes of four
__device__ __forceinline__ uint32_t bytes4(float x, float y, float z, float w) {
  return __byte_perm(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x0040),
                     __byte_perm(__float_as_uint(z), __float_as_uint(w), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t codes4(uint64_t a, uint64_t b, float inv) {
  const float2 x = unpack2(code_bits(a, inv)), y = unpack2(code_bits(b, inv));
  return bytes4(x.x, x.y, y.x, y.y);
}
// byte i of c as its code: the byte under the exponent of 2^23, minus 2^23 + 128
__device__ __forceinline__ float code_value(uint32_t c, int i) {
  return __uint_as_float(__byte_perm(c, 0x4b000000u, 0x7550 | i)) - 8388736.f;
}
// codes at scale s_old as codes at a larger scale, r = s_old / s
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float r) {
  return codes4(pack2(code_value(c, 0), code_value(c, 1)), pack2(code_value(c, 2), code_value(c, 3)), r);
}

// The page that a CTA works on and its new rows; valid: there are any.
struct PageTask {
  int page_index;
  int first, last;  // slots [first, last) of the page take new rows
  int pos0, row0;   // position and packed row of slot `first`
  bool valid;
};
__device__ __forceinline__ PageTask page_task(const Kv8View& c, const Kv8Batch& q, int b, int k) {
  PageTask t;
  const Kv8Session s = kv8_session(q, b, c.max_context, c.err);
  t.page_index = s.L / kPage + k;
  const int lo = max(s.L, t.page_index * kPage), hi = min(s.L + s.n, (t.page_index + 1) * kPage);
  t.valid = s.n > 0 && lo < hi;
  t.first = lo - t.page_index * kPage;
  t.last = hi - t.page_index * kPage;
  t.pos0 = lo;
  t.row0 = s.r0 + lo - s.L;
  return t;
}
// The page's id, or -1 with the error word set.
__device__ __forceinline__ int page_id(const Kv8View& c, const Kv8Batch& q, int b, int page_index) {
  const int page = q.bt[(size_t)b * q.bt_stride + page_index];
  if (page >= 0 && page < c.pool_pages) return page;
  set_err(c.err, QTTS_DEV_BAD_PAGE);
  return -1;
}

// A block's new scale, from its new values' largest magnitude (as bits).
__device__ __forceinline__ float new_scale(uint32_t amax, float s_old) {
  float s = __uint_as_float(amax) / 127.f;
  if (s < kKv8MinScale) s = 0.f;
  if (amax >= 0x7f800000u || s_old != s_old) s = __int_as_float(0x7fffffff);
  return s_old > s ? s_old : s;
}

// Append: one warp per block, the rows that it adds to the block in registers (of
// which three spill at head_dim 128): read them once, rotate (K), take the block's
// largest magnitude, quantise, write. Bound by bytes for prompts and by latency for single tokens, so the
// rows are asked for as soon as the session's lengths are there, together with
// the page's id and the rotation (once per CTA, in shared memory). 32 sessions of
// 60 to 1000 tokens, 8 kv heads of 128 (105 MB): 30 us, 3.5 TB/s, where the
// bytes would allow 15.5; the other half goes to instructions (K is rotated twice) and
// to the phases of a CTA (lengths, rows, codes). One token of 32 sessions: 4 us.
template <int D>
__global__ void __launch_bounds__(kMaxWarps * 32, 2)
    append_kernel(Kv8View c, Kv8Batch q, int touched, const uint16_t* __restrict__ k, int64_t k_stride,
                  const uint16_t* __restrict__ v, int64_t v_stride) {
  __shared__ __align__(16) float cs[kPage][D / 2], sn[kPage][D / 2], neg[kPage][D / 2];  // neg: -sn
  grid_dependency_wait();
  const int b = blockIdx.x / touched;
  const PageTask t = page_task(c, q, b, blockIdx.x % touched);
  if (!t.valid) return;
  const int lane = threadIdx.x & 31, task = blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;
  const bool active = task < 2 * c.nkv;
  const int h = task >> 1, which = task & 1;  // K, V

  // K: lanes of a token take dims 4i..4i+3 and their rotation partners d/2
  // further. V: a lane takes 4 dims of the tokens of NQ quads. 16 words either way
  constexpr int LPT = D / 8, TPP = 32 / LPT, PASSES = kPage / TPP;
  constexpr int NQ = D / 32, WORDS = 4 * NQ;
  static_assert(2 * PASSES == WORDS, "K and V words of a lane");
  const int i4 = lane % LPT * 4, tk = lane / LPT;                    // K
  const int x4 = lane % (D / 4), t0 = lane / (D / 4) * NQ;           // V
  auto v_slot = [&](int n, int j) { return 2 * (t0 + n) + (j & 1) + (j >> 1) * 8; };
  const bool all = t.first == 0 && t.last == kPage;
  auto fresh_slot = [&](int slot) { return all || (slot >= t.first && slot < t.last); };
  uint2 raw[WORDS];
  if (active && which == 0) {
    const uint16_t* src = k + (int64_t)(t.row0 - t.first + tk) * k_stride + h * D + i4;
#pragma unroll
    for (int p = 0; p < PASSES; ++p, src += TPP * k_stride) {
      raw[2 * p] = raw[2 * p + 1] = make_uint2(0u, 0u);
      if (fresh_slot(p * TPP + tk)) {
        raw[2 * p] = __ldcs((const uint2*)src);
        raw[2 * p + 1] = __ldcs((const uint2*)(src + D / 2));
      }
    }
  } else if (active) {
    const uint16_t* src = v + (int64_t)(t.row0 - t.first + 2 * t0) * v_stride + h * D + x4 * 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n, src += 2 * v_stride)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[4 * n + j] = make_uint2(0u, 0u);
        if (fresh_slot(v_slot(n, j))) raw[4 * n + j] = __ldcs((const uint2*)(src + ((j & 1) + (j >> 1) * 8) * v_stride));
      }
  }
  const int page = page_id(c, q, b, t.page_index);
  if (c.rope_cos) {
    const int n4 = (t.last - t.first) * (D / 8);  // float4s of each table
    const float4* c4 = (const float4*)(c.rope_cos + (size_t)t.pos0 * (D / 2));
    const float4* s4 = (const float4*)(c.rope_sin + (size_t)t.pos0 * (D / 2));
    for (int i = threadIdx.x; i < n4; i += blockDim.x) {
      ((float4*)cs[t.first])[i] = c4[i];
      const float4 v = s4[i];
      ((float4*)sn[t.first])[i] = v;
      ((float4*)neg[t.first])[i] = make_float4(-v.x, -v.y, -v.z, -v.w);
    }
    __syncthreads();
  }
  if (!active || page < 0) return;

  const size_t blk = (size_t)page * c.nkv + h;
  uint8_t* codes = c.codes + blk * (32 * D) + which * (16 * D);
  float* sp = c.scales + blk * 2 + which;
  // the tokens before the first new slot stay; their scale counts
  const float s_old = t.first > 0 ? *sp : 0.f;

  if (which == 0) {
    // Rotated twice, for the magnitude and for the codes: kept, the values would
    // not fit the registers that two CTAs of 16 warps leave.
    auto rotated = [&](int p, uint64_t (&x)[2], uint64_t (&y)[2]) {
      const int slot = p * TPP + tk;
      bf4(raw[2 * p], x[0], x[1]);
      bf4(raw[2 * p + 1], y[0], y[1]);
      if (c.rope_cos) {
        const ulonglong2 f = *(const ulonglong2*)&cs[slot][i4], g = *(const ulonglong2*)&sn[slot][i4],
                         h = *(const ulonglong2*)&neg[slot][i4];
        const uint64_t u0 = x[0], u1 = x[1];
        x[0] = fma2(u0, f.x, mul2(y[0], h.x));
        x[1] = fma2(u1, f.y, mul2(y[1], h.y));
        y[0] = fma2(y[0], f.x, mul2(u0, g.x));
        y[1] = fma2(y[1], f.y, mul2(u1, g.y));
      }
    };
    // dims x of token `slot` stand at [x / 64][slot][x % 64]
    uint8_t* dst = codes + i4 / 64 * 1024 + i4 % 64 + tk * 64;
    constexpr int kPartner = D == 128 ? 1024 : 32;
    auto block = [&](auto fresh) {
      float mx = 0.f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (fresh(p * TPP + tk)) {
          uint64_t x[2], y[2];
          rotated(p, x, y);
          mx = max_abs(max_abs(max_abs(max_abs(mx, x[0]), x[1]), y[0]), y[1]);
        }
      const float s = new_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)), s_old);
      const float inv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
      for (int p = 0; p < WORDS; ++p) asm volatile("" : "+r"(raw[p].x), "+r"(raw[p].y));  // or the compiler keeps them
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (fresh(p * TPP + tk)) {
          uint64_t x[2], y[2];
          rotated(p, x, y);
          *(uint32_t*)(dst + p * TPP * 64) = codes4(x[0], x[1], inv);
          *(uint32_t*)(dst + p * TPP * 64 + kPartner) = codes4(y[0], y[1], inv);
        }
      return s;
    };
    float s;
    if (all) {
      s = block([](int) { return true; });
    } else {
      s = block([&](int slot) { return slot >= t.first && slot < t.last; });
      if (s > s_old && s_old > 0.f) {  // the codes of the tokens before follow
        const float r = s_old / s;
#pragma unroll 1
        for (int p = 0; p * TPP + tk < t.first; ++p) {
          uint32_t* w = (uint32_t*)(dst + p * TPP * 64);
          uint32_t* v = (uint32_t*)(dst + p * TPP * 64 + kPartner);
          *w = rescale4(*w, r);
          *v = rescale4(*v, r);
        }
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *sp = s;
  } else {
    uint32_t mx = 0;  // two magnitudes as 16-bit halves
#pragma unroll
    for (int p = 0; p < WORDS; ++p) mx = __vmaxu2(mx, __vmaxu2(raw[p].x & 0x7fff7fffu, raw[p].y & 0x7fff7fffu));
    mx = max(mx & 0xffffu, mx >> 16) << 16;
    const float s = new_scale(__reduce_max_sync(0xffffffffu, mx), s_old);
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const bool grown = s > s_old && s_old > 0.f;
    const float r = grown ? s_old / s : 0.f;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      uint4* dst = (uint4*)(codes + x4 * 64 + (t0 + n) * 16);
      float2 q[4][2];  // token j's four codes
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t a, b;
        bf4(raw[4 * n + j], a, b);
        q[j][0] = unpack2(code_bits(a, inv));
        q[j][1] = unpack2(code_bits(b, inv));
      }
      // word i: dim 4 x4 + i, byte j: token j of the quad
      uint4 o = make_uint4(bytes4(q[0][0].x, q[1][0].x, q[2][0].x, q[3][0].x), bytes4(q[0][0].y, q[1][0].y, q[2][0].y, q[3][0].y),
                           bytes4(q[0][1].x, q[1][1].x, q[2][1].x, q[3][1].x), bytes4(q[0][1].y, q[1][1].y, q[2][1].y, q[3][1].y));
      if (!all) {
        uint4 old = *dst;
        uint32_t fresh = 0, before = 0;  // byte masks of the new tokens, of those before them
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (v_slot(n, j) >= t.first && v_slot(n, j) < t.last) fresh |= 255u << (8 * j);
          if (v_slot(n, j) < t.first) before |= 255u << (8 * j);
        }
        if (!grown) before = 0;
        auto merge = [&](uint32_t now, uint32_t was) {
          if (before) was = (was & ~before) | (rescale4(was, r) & before);
          return (now & fresh) | (was & ~fresh);
        };
        o = make_uint4(merge(o.x, old.x), merge(o.y, old.y), merge(o.z, old.z), merge(o.w, old.w));
      }
      *dst = o;
    }
    __syncwarp();
    if (lane == 0) *sp = s;
  }
}

// Read-back: codes times scale as bf16, one warp per block, rows packed. Bound by
// bytes: 18 us for the 105 MB above, 5.8 TB/s.
template <int D>
__global__ void __launch_bounds__(kMaxWarps * 32, 4)
    read_kernel(Kv8View c, Kv8Batch q, int touched, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  grid_dependency_wait();
  const int b = blockIdx.x / touched;
  const PageTask t = page_task(c, q, b, blockIdx.x % touched);
  const int lane = threadIdx.x & 31, task = blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;
  if (!t.valid || task >= 2 * c.nkv) return;
  const int h = task >> 1, which = task & 1;
  const int page = page_id(c, q, b, t.page_index);
  if (page < 0) return;
  const size_t blk = (size_t)page * c.nkv + h;
  const uint8_t* codes = c.codes + blk * (32 * D) + which * (16 * D);
  const float s = c.scales[blk * 2 + which];
  const bool all = t.first == 0 && t.last == kPage;
  auto wanted = [&](int slot) { return all || (slot >= t.first && slot < t.last); };
  const int64_t pitch = (int64_t)c.nkv * D;
  auto pair = [&](uint32_t w0, int i0, uint32_t w1, int i1) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(code_value(w0, i0) * s, code_value(w1, i1) * s);
    return *(const uint32_t*)&p;
  };
  if (which == 0) {
    constexpr int LPT = D / 4, TPP = 32 / LPT, PASSES = kPage / TPP;
    const int x = lane % LPT * 4;
    uint32_t w[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) w[p] = *(const uint32_t*)(codes + x / 64 * 1024 + (p * TPP + lane / LPT) * 64 + x % 64);
    uint16_t* o = k + (t.row0 - t.first + lane / LPT) * pitch + h * D + x;
#pragma unroll
    for (int p = 0; p < PASSES; ++p, o += TPP * pitch)
      if (wanted(p * TPP + lane / LPT))
        __stcs((uint2*)o, make_uint2(pair(w[p], 0, w[p], 1), pair(w[p], 2, w[p], 3)));
  } else {
    constexpr int NQ = D / 32;
    const int x4 = lane % (D / 4), t0 = lane / (D / 4) * NQ;
    uint4 w[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) w[n] = *(const uint4*)(codes + x4 * 64 + (t0 + n) * 16);
    uint16_t* o = v + (t.row0 - t.first + 2 * t0) * pitch + h * D + x4 * 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n, o += 2 * pitch)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (wanted(2 * (t0 + n) + (j & 1) + (j >> 1) * 8))
          __stcs((uint2*)(o + ((j & 1) + (j >> 1) * 8) * pitch),
                 make_uint2(pair(w[n].x, j, w[n].y, j), pair(w[n].z, j, w[n].w, j)));
  }
}

thread_local ErrorText g_err;  // of calls without a handle

int fail(qtts_kv8* c, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  (c ? c->err : g_err).set(fmt, ap);
  va_end(ap);
  return code;
}

// A failed runtime call is reported here, not by a later call's check of the last error.
int cuda_fault(qtts_kv8* c, const char* who, cudaError_t e) {
  cudaGetLastError();
  return fail(c, e == cudaErrorMemoryAllocation ? QTTS_E_OOM : QTTS_E_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

const char* config_fault(const qtts_kv8_config& c) {
  if (c.n_layers <= 0 || c.n_q_heads <= 0 || c.n_kv_heads <= 0 || c.pool_pages <= 0) return "sizes must be positive";
  if (c.head_dim != 64 && c.head_dim != 128) return "head_dim must be 64 or 128";
  if (c.n_kv_heads > 1024) return "at most 1024 kv heads";
  if (c.n_q_heads % c.n_kv_heads) return "q heads % kv heads != 0";
  if (c.n_q_heads / c.n_kv_heads > kKv8MaxGroup) return "at most 32 q heads per kv head";
  if (c.page_size != kPage) return "page_size must be 16";
  if (c.max_batch <= 0 || c.max_batch > kKv8MaxBatch) return "max_batch must be in 1..1024";
  if (c.max_context <= 0 || c.max_context > kKv8MaxContext) return "max_context must be in 1..262144";
  if (!(c.rope_theta >= 0.f) || std::isinf(c.rope_theta)) return "rope_theta must be finite and not negative";
  if ((long long)c.pool_pages * c.n_kv_heads > 0x7fffffffll) return "pool_pages x n_kv_heads must be below 2^31";
  // bytes of the codes stay countable (an allocation of 2^52 fails, one of 2^64 would be taken for 0)
  if ((long long)c.pool_pages * c.n_kv_heads > (1ll << 40) / c.n_layers) return "n_layers x pool_pages x n_kv_heads must be at most 2^40";
  return nullptr;
}

// The checks that append, attention and read share. Returns a negative code,
// 0 (go on), or 1 (nothing to do).
int check_batch(qtts_kv8* c, const char* who, int layer, const Kv8Batch& q) {
  const qtts_kv8_config& f = c->cfg;
  if (layer < 0 || layer >= f.n_layers) return fail(c, QTTS_E_INVALID, "%s: layer %d outside 0..%d", who, layer, f.n_layers - 1);
  if (q.B < 1 || q.B > f.max_batch) return fail(c, QTTS_E_BATCH, "%s: B = %d outside 1..%d", who, q.B, f.max_batch);
  if (q.n_rows < 0 || q.max_new < 1 || q.bt_stride < 1) return fail(c, QTTS_E_INVALID, "%s: bad row count or table stride", who);
  if (!q.row_start && (q.n_rows != q.B || q.max_new != 1))
    return fail(c, QTTS_E_INVALID, "%s: without row_start there is one row per session", who);
  if (!q.kv_len || !q.bt) return fail(c, QTTS_E_INVALID, "%s: null argument", who);
  return q.n_rows == 0 ? 1 : 0;
}
bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && ((uintptr_t)p & 7) == 0 && stride >= width && stride % 4 == 0;
}

Kv8View view(const qtts_kv8* c, int layer) {
  const qtts_kv8_config& f = c->cfg;
  const size_t blocks = (size_t)f.pool_pages * f.n_kv_heads * layer;
  return {c->codes + blocks * 32 * f.head_dim, c->scales + blocks * 2, c->rope_cos, c->rope_sin, f.n_kv_heads,
          f.pool_pages, f.max_context, c->dev_err};
}
// Pages that a session's rows can touch, wherever they start. max_new and n_rows are
// bounds that a caller may set as high as it likes; a session ends at max_context.
int touched_pages(int max_new, int n_rows, int max_context) {
  return (std::min({max_new, n_rows, max_context}) + 2 * kPage - 2) / kPage;
}
static_assert((kKv8MaxContext + 2 * kPage) / kPage * (long long)kKv8MaxBatch <= 0x7fffffff, "CTAs of a grid");

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.stream = s;
  cudaLaunchAttribute at[1];
  early_launch(lc, at);
  return cudaLaunchKernelEx(&lc, kern, (P)args...);
}

}  // namespace
}  // namespace qtts

using namespace qtts;

extern "C" {

const char* qtts_kv8_last_error(const qtts_kv8* c) { return (c ? c->err : g_err).get(); }

int qtts_kv8_create(const qtts_kv8_config* cfg, int device, qtts_kv8** out) {
  if (!cfg || !out) return fail(nullptr, QTTS_E_INVALID, "null argument");
  *out = nullptr;
  if (const char* why = config_fault(*cfg)) return fail(nullptr, QTTS_E_INVALID, "bad config: %s", why);
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) cudaGetLastError();
  if (device < 0 || device >= ndev) return fail(nullptr, QTTS_E_CUDA, "no CUDA device %d", device);
  DeviceGuard g(device);
  if (!g.ok) return fail(nullptr, QTTS_E_CUDA, "cudaSetDevice(%d) failed", device);
  qtts_kv8* c = new (std::nothrow) qtts_kv8();
  if (!c) return fail(nullptr, QTTS_E_OOM, "out of host memory");
  auto bail = [&](const char* what, cudaError_t e) {
    qtts_kv8_destroy(c);
    return cuda_fault(nullptr, what, e);
  };
  c->cfg = *cfg;
  c->device = device;
  try {
    c->page_used.assign(cfg->pool_pages, 0);
    c->seen_now.assign(cfg->pool_pages, 0);
    c->free_ids.resize(cfg->pool_pages);
  } catch (const std::bad_alloc&) {
    return bail("page list", cudaErrorMemoryAllocation);
  }
  for (int i = 0; i < cfg->pool_pages; ++i) c->free_ids[i] = cfg->pool_pages - 1 - i;  // handed out 0, 1, 2, ...
  cudaError_t e = cudaDeviceGetAttribute(&c->G, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = kv8_attention_setup(cfg->head_dim);
  if (e != cudaSuccess) return bail("kernel setup", e);
  const size_t blocks = (size_t)cfg->n_layers * cfg->pool_pages * cfg->n_kv_heads;
  const size_t half = cfg->head_dim / 2, table = (size_t)cfg->max_context * half * sizeof(float);
  e = cudaMalloc((void**)&c->codes, blocks * 32 * cfg->head_dim);
  if (e == cudaSuccess) e = cudaMalloc((void**)&c->scales, blocks * 2 * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc((void**)&c->dev_err, sizeof(int));
  if (e == cudaSuccess && cfg->rope_theta > 0.f) e = cudaMalloc((void**)&c->rope_cos, table);
  if (e == cudaSuccess && cfg->rope_theta > 0.f) e = cudaMalloc((void**)&c->rope_sin, table);
  if (e != cudaSuccess) return bail("device allocation", e);
  // pages start as zero scales: a page that was never appended to reads as 0
  e = cudaMemset(c->scales, 0, blocks * 2 * sizeof(float));
  if (e == cudaSuccess) e = cudaMemset(c->codes, 128, blocks * 32 * cfg->head_dim);
  if (e == cudaSuccess) e = cudaMemset(c->dev_err, 0, sizeof(int));
  if (e == cudaSuccess && c->rope_cos)
    e = launch(rope_table_kernel, dim3(std::min(cfg->max_context, 4096)), (int)half, nullptr, c->rope_cos, c->rope_sin,
               cfg->max_context, (int)half, (double)cfg->rope_theta);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return bail("cache setup", e);
  *out = c;
  return QTTS_OK;
}

void qtts_kv8_destroy(qtts_kv8* c) {
  if (!c) return;
  {
    DeviceGuard g(c->device);
    for (void* p : {(void*)c->codes, (void*)c->scales, (void*)c->rope_cos, (void*)c->rope_sin, (void*)c->dev_err})
      if (p && cudaFree(p) != cudaSuccess) cudaGetLastError();
  }
  delete c;
}

int qtts_kv8_alloc_pages(qtts_kv8* c, int n, int32_t* ids) {
  if (!c || n < 0 || (n && !ids)) return fail(c, QTTS_E_INVALID, "bad argument");
  if ((size_t)n > c->free_ids.size())
    return fail(c, QTTS_E_POOL, "KV pool has %zu free pages, %d requested", c->free_ids.size(), n);
  for (int i = 0; i < n; ++i) {
    ids[i] = c->free_ids.back();
    c->free_ids.pop_back();
    c->page_used[ids[i]] = 1;
  }
  return QTTS_OK;
}

int qtts_kv8_free_pages(qtts_kv8* c, int n, const int32_t* ids) {
  if (!c || n < 0 || (n && !ids)) return fail(c, QTTS_E_INVALID, "bad argument");
  int bad = n;
  for (int i = 0; i < n && bad == n; ++i) {
    if (ids[i] < 0 || ids[i] >= c->cfg.pool_pages || !c->page_used[ids[i]] || c->seen_now[ids[i]]) bad = i;
    else c->seen_now[ids[i]] = 1;
  }
  for (int i = 0; i < bad; ++i) c->seen_now[ids[i]] = 0;
  if (bad < n) return fail(c, QTTS_E_POOL, "page %d is not allocated", ids[bad]);
  for (int i = 0; i < n; ++i) {
    c->page_used[ids[i]] = 0;
    c->free_ids.push_back(ids[i]);  // within the capacity reserved at creation
  }
  return QTTS_OK;
}

int qtts_kv8_free_count(const qtts_kv8* c) { return c ? (int)c->free_ids.size() : 0; }

int64_t qtts_kv8_workspace_bytes(const qtts_kv8* c) {
  return c ? (int64_t)kv8_attention_workspace(c->cfg.head_dim, c->G) : 0;
}

int qtts_kv8_append(qtts_kv8* c, int layer, int B, int n_rows, int max_new, const int32_t* row_start,
                    const int32_t* kv_len, const int32_t* block_tables, int bt_stride, const uint16_t* k,
                    int64_t k_stride, const uint16_t* v, int64_t v_stride, void* stream) {
  if (!c) return QTTS_E_INVALID;
  const Kv8Batch q{B, n_rows, max_new, row_start, kv_len, block_tables, bt_stride};
  const int rc = check_batch(c, "qtts_kv8_append", layer, q);
  if (rc < 0) return rc;
  const qtts_kv8_config& f = c->cfg;
  const int64_t width = (int64_t)f.n_kv_heads * f.head_dim;
  if (rc == 0 && (!rows_ok(k, k_stride, width) || !rows_ok(v, v_stride, width)))
    return fail(c, QTTS_E_INVALID,
                "qtts_kv8_append: k and v must be 8-byte aligned, with row strides that are multiples of 4 and hold a row");
  if (rc) return QTTS_OK;
  DeviceGuard g(c->device);
  if (!g.ok) return fail(c, QTTS_E_CUDA, "cudaSetDevice failed");
  const int touched = touched_pages(max_new, n_rows, f.max_context);
  const int warps = std::min(2 * f.n_kv_heads, kMaxWarps);
  const dim3 grid(B * touched, (2 * f.n_kv_heads + warps - 1) / warps);
  const cudaError_t e = launch(f.head_dim == 64 ? append_kernel<64> : append_kernel<128>, grid, warps * 32,
                               (cudaStream_t)stream, view(c, layer), q, touched, k, k_stride, v, v_stride);
  if (e != cudaSuccess) return cuda_fault(c, "qtts_kv8_append", e);
  return QTTS_OK;
}

int qtts_kv8_read(qtts_kv8* c, int layer, int B, int n_rows, int max_new, const int32_t* row_start,
                  const int32_t* pos0, const int32_t* block_tables, int bt_stride, uint16_t* k_out, uint16_t* v_out,
                  void* stream) {
  if (!c) return QTTS_E_INVALID;
  const Kv8Batch q{B, n_rows, max_new, row_start, pos0, block_tables, bt_stride};
  const int rc = check_batch(c, "qtts_kv8_read", layer, q);
  if (rc < 0) return rc;
  const qtts_kv8_config& f = c->cfg;
  const int64_t width = (int64_t)f.n_kv_heads * f.head_dim;
  if (rc == 0 && (!rows_ok(k_out, width, width) || !rows_ok(v_out, width, width)))
    return fail(c, QTTS_E_INVALID, "qtts_kv8_read: k_out and v_out must be 8-byte aligned");
  if (rc) return QTTS_OK;
  DeviceGuard g(c->device);
  if (!g.ok) return fail(c, QTTS_E_CUDA, "cudaSetDevice failed");
  const int touched = touched_pages(max_new, n_rows, f.max_context);
  const int warps = std::min(2 * f.n_kv_heads, kMaxWarps);
  const dim3 grid(B * touched, (2 * f.n_kv_heads + warps - 1) / warps);
  const cudaError_t e = launch(f.head_dim == 64 ? read_kernel<64> : read_kernel<128>, grid, warps * 32,
                               (cudaStream_t)stream, view(c, layer), q, touched, k_out, v_out);
  if (e != cudaSuccess) return cuda_fault(c, "qtts_kv8_read", e);
  return QTTS_OK;
}

int qtts_kv8_attention(qtts_kv8* c, int layer, int B, int n_rows, int max_new, const int32_t* row_start,
                       const int32_t* kv_len, const int32_t* block_tables, int bt_stride, const uint16_t* q,
                       int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, void* workspace,
                       void* stream) {
  if (!c) return QTTS_E_INVALID;
  const Kv8Batch qb{B, n_rows, max_new, row_start, kv_len, block_tables, bt_stride};
  const int rc = check_batch(c, "qtts_kv8_attention", layer, qb);
  if (rc < 0) return rc;
  const qtts_kv8_config& f = c->cfg;
  const int64_t width = (int64_t)f.n_q_heads * f.head_dim;
  if (rc == 0 && (!rows_ok(q, q_stride, width) || !rows_ok(out, out_stride, width)))
    return fail(c, QTTS_E_INVALID,
                "qtts_kv8_attention: q and out must be 8-byte aligned, with row strides that are multiples of 4 and hold a row");
  if (rc == 0 && (!workspace || ((uintptr_t)workspace & 15)))
    return fail(c, QTTS_E_INVALID, "qtts_kv8_attention: workspace must be given and 16-byte aligned");
  if (!std::isfinite(scale)) return fail(c, QTTS_E_INVALID, "qtts_kv8_attention: scale must be finite");
  if (rc) return QTTS_OK;
  if (!kv8_attention_fits(view(c, layer), qb, f.n_q_heads / f.n_kv_heads))
    return fail(c, QTTS_E_INVALID, "qtts_kv8_attention: too much work for one call, split the batch");
  DeviceGuard g(c->device);
  if (!g.ok) return fail(c, QTTS_E_CUDA, "cudaSetDevice failed");
  const cudaError_t e = kv8_attention(view(c, layer), qb, f.head_dim, f.n_q_heads / f.n_kv_heads, c->G, q, q_stride,
                                      scale, out, out_stride, workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fault(c, "qtts_kv8_attention", e);
  return QTTS_OK;
}

int qtts_kv8_status(qtts_kv8* c, int* device_err) {
  if (device_err) *device_err = QTTS_DEV_OK;
  if (!c) return QTTS_E_INVALID;
  DeviceGuard g(c->device);
  if (!g.ok) return fail(c, QTTS_E_CUDA, "cudaSetDevice failed");
  int v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, c->dev_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) {
    // waited for: other streams do not wait for it, and their errors are the next call's
    e = cudaMemset(c->dev_err, 0, sizeof(int));
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  }
  if (e != cudaSuccess) return cuda_fault(c, "qtts_kv8_status", e);
  if (device_err) *device_err = v;
  if (v == QTTS_DEV_TIMEOUT) return fail(c, QTTS_E_TIMEOUT, "a device-side wait ran out its limit");
  if (v) return fail(c, QTTS_E_DEVICE, "device-side check failed: %d", v);
  return QTTS_OK;
}

}  // extern "C"
