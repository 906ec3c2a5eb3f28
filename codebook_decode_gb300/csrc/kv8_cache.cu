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

constexpr int kWarpsPerCta = 4;  // one warp per (page, head, K or V) block

// The rotation table: angles in double (a position of a long context times a
// frequency loses its fraction in fp32), stored fp32.
__global__ void rope_table_kernel(float* cs, float* sn, int max_context, int half, double theta) {
  const int i = threadIdx.x;
  const double f = pow(theta, -(double)i / half);
  for (int p = blockIdx.x; p < max_context; p += gridDim.x) {
    double s, c;
    sincos((double)p * f, &s, &c);
    cs[(size_t)p * half + i] = (float)c;
    sn[(size_t)p * half + i] = (float)s;
  }
}

__device__ __forceinline__ float4 bf4(uint2 v) {
  return make_float4(bf2f(v.x & 0xffffu), __uint_as_float(v.x & 0xffff0000u), bf2f(v.y & 0xffffu),
                     __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ uint32_t abs_bits4(float4 v) {
  const uint32_t m = 0x7fffffffu;
  return max(max(__float_as_uint(v.x) & m, __float_as_uint(v.y) & m),
             max(__float_as_uint(v.z) & m, __float_as_uint(v.w) & m));
}
__device__ __forceinline__ uint32_t code(float x, float inv) {
  return (uint32_t)(__float2int_rn(fminf(fmaxf(x * inv, -127.f), 127.f)) + 128);
}
__device__ __forceinline__ uint32_t codes4(float4 v, float inv) {
  return code(v.x, inv) | code(v.y, inv) << 8 | code(v.z, inv) << 16 | code(v.w, inv) << 24;
}
// codes at scale s_old as codes at a larger scale, r = s_old / s
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float r) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= code((float)((int)(c >> (8 * i) & 255u) - 128), r) << (8 * i);
  return o;
}

struct BlockTask {
  int b, page, h, which;  // which: 0 K, 1 V
  int first, last;        // slots [first, last) of the page take new rows
  int pos0, row0;         // position and packed row of slot `first`
};
// The block that this warp works on; false: none, or a page outside the pool.
__device__ __forceinline__ bool block_task(const Kv8View& c, const Kv8Batch& q, int touched, BlockTask* t) {
  t->b = blockIdx.x / touched;
  const int k = blockIdx.x % touched;
  const int task = blockIdx.y * kWarpsPerCta + threadIdx.x / 32;
  if (task >= 2 * c.nkv) return false;
  t->h = task >> 1;
  t->which = task & 1;
  const Kv8Session s = kv8_session(q, t->b, c.max_context, c.err);
  if (s.n == 0) return false;
  const int pi = s.L / kPage + k;
  const int lo = max(s.L, pi * kPage), hi = min(s.L + s.n, (pi + 1) * kPage);
  if (lo >= hi) return false;
  t->page = q.bt[(size_t)t->b * q.bt_stride + pi];
  if (t->page < 0 || t->page >= c.pool_pages) {
    set_err(c.err, QTTS_DEV_BAD_PAGE);
    return false;
  }
  t->first = lo - pi * kPage;
  t->last = hi - pi * kPage;
  t->pos0 = lo;
  t->row0 = s.r0 + lo - s.L;
  return true;
}

// Append: one warp per block, everything it adds to the block in registers:
// read the rows once, rotate (K), take the block's largest magnitude, quantise,
// write. Rows are read 8 bytes a lane (a token's head is 256 contiguous bytes
// at d = 128). Bound by bytes for prompts and by latency for single tokens.
template <int D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    append_kernel(Kv8View c, Kv8Batch q, int touched, const uint16_t* __restrict__ k, int64_t k_stride,
                  const uint16_t* __restrict__ v, int64_t v_stride) {
  BlockTask t;
  if (!block_task(c, q, touched, &t)) return;
  const int lane = threadIdx.x & 31;
  const size_t blk = (size_t)t.page * c.nkv + t.h;
  uint8_t* codes = c.codes + blk * (32 * D) + t.which * (16 * D);
  float* sp = c.scales + blk * 2 + t.which;
  // the tokens before the first new slot stay; their scale counts
  const float s_old = t.first > 0 ? *sp : 0.f;
  uint32_t amax = 0;

  if (t.which == 0) {
    // lanes of a token take dims 4i..4i+3 and their rotation partners d/2 further
    constexpr int LPT = D / 8, TPP = 32 / LPT, PASSES = kPage / TPP;
    const int i4 = lane % LPT * 4, tk = lane / LPT;
    float4 a[PASSES], b[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int slot = p * TPP + tk;
      a[p] = b[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (slot >= t.first && slot < t.last) {
        const uint16_t* row = k + (int64_t)(t.row0 + slot - t.first) * k_stride + t.h * D + i4;
        a[p] = bf4(*(const uint2*)row);
        b[p] = bf4(*(const uint2*)(row + D / 2));
      }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int slot = p * TPP + tk;
      if (c.rope_cos && slot >= t.first && slot < t.last) {
        const size_t at = (size_t)(t.pos0 + slot - t.first) * (D / 2) + i4;
        const float4 cs = *(const float4*)(c.rope_cos + at), sn = *(const float4*)(c.rope_sin + at);
        const float4 x = a[p], y = b[p];
        a[p] = make_float4(x.x * cs.x - y.x * sn.x, x.y * cs.y - y.y * sn.y, x.z * cs.z - y.z * sn.z,
                           x.w * cs.w - y.w * sn.w);
        b[p] = make_float4(y.x * cs.x + x.x * sn.x, y.y * cs.y + x.y * sn.y, y.z * cs.z + x.z * sn.z,
                           y.w * cs.w + x.w * sn.w);
      }
      amax = max(amax, max(abs_bits4(a[p]), abs_bits4(b[p])));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    float s = __uint_as_float(amax) / 127.f;
    if (s < kKv8MinScale) s = 0.f;
    if (amax >= 0x7f800000u || s_old != s_old) s = __int_as_float(0x7fffffff);
    if (s_old > s) s = s_old;
    const float inv = s > 0.f ? 1.f / s : 0.f;
    // dims x of token `slot` stand at [x / 64][slot][x % 64]
    auto at = [&](int slot, int x) { return (uint32_t*)(codes + x / 64 * 1024 + slot * 64 + x % 64); };
    const bool grown = s > s_old && s_old > 0.f;
    const float r = grown ? s_old / s : 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int slot = p * TPP + tk;
      if (slot >= t.first && slot < t.last) {
        *at(slot, i4) = codes4(a[p], inv);
        *at(slot, i4 + D / 2) = codes4(b[p], inv);
      } else if (grown && slot < t.first) {
        *at(slot, i4) = rescale4(*at(slot, i4), r);
        *at(slot, i4 + D / 2) = rescale4(*at(slot, i4 + D / 2), r);
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *sp = s;
  } else {
    // a lane takes 4 dims of the tokens of NQ quads: 16-byte words of 4 dims x 4 tokens
    constexpr int NQ = D / 32;
    const int x4 = lane % (D / 4), t0 = lane / (D / 4) * NQ;
    float4 a[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = 2 * (t0 + n) + (j & 1) + (j >> 1) * 8;
        a[n][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (slot >= t.first && slot < t.last)
          a[n][j] = bf4(*(const uint2*)(v + (int64_t)(t.row0 + slot - t.first) * v_stride + t.h * D + x4 * 4));
        amax = max(amax, abs_bits4(a[n][j]));
      }
    amax = __reduce_max_sync(0xffffffffu, amax);
    float s = __uint_as_float(amax) / 127.f;
    if (s < kKv8MinScale) s = 0.f;
    if (amax >= 0x7f800000u || s_old != s_old) s = __int_as_float(0x7fffffff);
    if (s_old > s) s = s_old;
    const float inv = s > 0.f ? 1.f / s : 0.f;
    const bool whole = t.first == 0 && t.last == kPage;
    const bool grown = s > s_old && s_old > 0.f;
    const float r = grown ? s_old / s : 0.f;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      uint4* w = (uint4*)(codes + x4 * 64 + (t0 + n) * 16);
      uint4 o = make_uint4(0, 0, 0, 0);
      if (!whole) o = *w;
      uint32_t* ow = &o.x;  // word i: dim 4 x4 + i, byte j: token j of the quad
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = 2 * (t0 + n) + (j & 1) + (j >> 1) * 8;
        if (slot >= t.first && slot < t.last) {
          const float* f = &a[n][j].x;
#pragma unroll
          for (int i = 0; i < 4; ++i) ow[i] = (ow[i] & ~(255u << (8 * j))) | code(f[i], inv) << (8 * j);
        } else if (grown && slot < t.first) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float old = (float)((int)(ow[i] >> (8 * j) & 255u) - 128);
            ow[i] = (ow[i] & ~(255u << (8 * j))) | code(old, r) << (8 * j);
          }
        }
      }
      *w = o;
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *sp = s;
  }
}

// Read-back: codes times scale as bf16, one warp per block, rows packed.
template <int D>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
    read_kernel(Kv8View c, Kv8Batch q, int touched, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  BlockTask t;
  if (!block_task(c, q, touched, &t)) return;
  const int lane = threadIdx.x & 31;
  const size_t blk = (size_t)t.page * c.nkv + t.h;
  const uint8_t* codes = c.codes + blk * (32 * D) + t.which * (16 * D);
  const float s = c.scales[blk * 2 + t.which];
  auto val = [&](uint32_t byte) { return (uint32_t)f2bf((float)((int)(byte & 255u) - 128) * s); };
  if (t.which == 0) {
    constexpr int LPT = D / 4, TPP = 32 / LPT;
    const int x = lane % LPT * 4;
#pragma unroll
    for (int p = 0; p < kPage / TPP; ++p) {
      const int slot = p * TPP + lane / LPT;
      if (slot < t.first || slot >= t.last) continue;
      const uint32_t w = *(const uint32_t*)(codes + x / 64 * 1024 + slot * 64 + x % 64);
      uint16_t* o = k + ((size_t)(t.row0 + slot - t.first) * c.nkv + t.h) * D + x;
      *(uint2*)o = make_uint2(val(w) | val(w >> 8) << 16, val(w >> 16) | val(w >> 24) << 16);
    }
  } else {
    constexpr int NQ = D / 32;
    const int x4 = lane % (D / 4), t0 = lane / (D / 4) * NQ;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const uint4 w = *(const uint4*)(codes + x4 * 64 + (t0 + n) * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = 2 * (t0 + n) + (j & 1) + (j >> 1) * 8;
        if (slot < t.first || slot >= t.last) continue;
        uint16_t* o = v + ((size_t)(t.row0 + slot - t.first) * c.nkv + t.h) * D + x4 * 4;
        *(uint2*)o = make_uint2(val(w.x >> (8 * j)) | val(w.y >> (8 * j)) << 16,
                                val(w.z >> (8 * j)) | val(w.w >> (8 * j)) << 16);
      }
    }
  }
}

char g_err[256];

int fail(qtts_kv8* c, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(c ? c->err : g_err, 256, fmt, ap);
  va_end(ap);
  return code;
}

// The caller's current device is put back on every path out.
struct DeviceGuard {
  int prev = -1, dev;
  bool ok;
  explicit DeviceGuard(int d) : dev(d) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    ok = prev == d || cudaSetDevice(d) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
};

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
// pages that max_new rows can touch, wherever they start
int touched_pages(int max_new) { return (max_new + 2 * kPage - 2) / kPage; }

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.stream = s;
  return cudaLaunchKernelEx(&lc, kern, (P)args...);
}

}  // namespace
}  // namespace qtts

using namespace qtts;

extern "C" {

const char* qtts_kv8_last_error(const qtts_kv8* c) { return c ? c->err : g_err; }

int qtts_kv8_create(const qtts_kv8_config* cfg, int device, qtts_kv8** out) {
  if (!cfg || !out) return fail(nullptr, QTTS_E_INVALID, "null argument");
  *out = nullptr;
  if (const char* why = config_fault(*cfg)) return fail(nullptr, QTTS_E_INVALID, "bad config: %s", why);
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev)
    return fail(nullptr, QTTS_E_CUDA, "no CUDA device %d", device);
  DeviceGuard g(device);
  if (!g.ok) return fail(nullptr, QTTS_E_CUDA, "cudaSetDevice(%d) failed", device);
  qtts_kv8* c = new (std::nothrow) qtts_kv8();
  if (!c) return fail(nullptr, QTTS_E_OOM, "out of host memory");
  auto bail = [&](int code, const char* what, cudaError_t e) {
    fail(nullptr, code, "%s: %s", what, cudaGetErrorString(e));
    qtts_kv8_destroy(c);
    return code;
  };
  c->cfg = *cfg;
  c->device = device;
  try {
    c->page_used.assign(cfg->pool_pages, 0);
    c->seen_now.assign(cfg->pool_pages, 0);
    c->free_ids.resize(cfg->pool_pages);
  } catch (const std::bad_alloc&) {
    return bail(QTTS_E_OOM, "page list", cudaErrorMemoryAllocation);
  }
  for (int i = 0; i < cfg->pool_pages; ++i) c->free_ids[i] = cfg->pool_pages - 1 - i;  // handed out 0, 1, 2, ...
  cudaError_t e = cudaDeviceGetAttribute(&c->G, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = kv8_attention_setup(cfg->head_dim);
  if (e != cudaSuccess) return bail(QTTS_E_CUDA, "kernel setup", e);
  const size_t blocks = (size_t)cfg->n_layers * cfg->pool_pages * cfg->n_kv_heads;
  const size_t half = cfg->head_dim / 2, table = (size_t)cfg->max_context * half * sizeof(float);
  e = cudaMalloc((void**)&c->codes, blocks * 32 * cfg->head_dim);
  if (e == cudaSuccess) e = cudaMalloc((void**)&c->scales, blocks * 2 * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc((void**)&c->dev_err, sizeof(int));
  if (e == cudaSuccess && cfg->rope_theta > 0.f) e = cudaMalloc((void**)&c->rope_cos, table);
  if (e == cudaSuccess && cfg->rope_theta > 0.f) e = cudaMalloc((void**)&c->rope_sin, table);
  if (e != cudaSuccess) {
    cudaGetLastError();  // the failed allocation's sticky-free error is reported here, not by a later call
    return bail(QTTS_E_OOM, "device allocation", e);
  }
  // pages start as zero scales: a page that was never appended to reads as 0
  e = cudaMemset(c->scales, 0, blocks * 2 * sizeof(float));
  if (e == cudaSuccess) e = cudaMemset(c->codes, 128, blocks * 32 * cfg->head_dim);
  if (e == cudaSuccess) e = cudaMemset(c->dev_err, 0, sizeof(int));
  if (e == cudaSuccess && c->rope_cos)
    e = launch(rope_table_kernel, dim3(std::min(cfg->max_context, 4096)), (int)half, nullptr, c->rope_cos, c->rope_sin,
               cfg->max_context, (int)half, (double)cfg->rope_theta);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return bail(QTTS_E_CUDA, "cache setup", e);
  *out = c;
  return QTTS_OK;
}

void qtts_kv8_destroy(qtts_kv8* c) {
  if (!c) return;
  {
    DeviceGuard g(c->device);
    for (void* p : {(void*)c->codes, (void*)c->scales, (void*)c->rope_cos, (void*)c->rope_sin, (void*)c->dev_err})
      if (p) cudaFree(p);
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
  const int touched = touched_pages(std::min(max_new, n_rows));
  if ((long long)B * touched > 0x7fffffffll) return fail(c, QTTS_E_INVALID, "qtts_kv8_append: too many rows");
  const dim3 grid(B * touched, (2 * f.n_kv_heads + kWarpsPerCta - 1) / kWarpsPerCta);
  const cudaError_t e = launch(f.head_dim == 64 ? append_kernel<64> : append_kernel<128>, grid, kWarpsPerCta * 32,
                               (cudaStream_t)stream, view(c, layer), q, touched, k, k_stride, v, v_stride);
  if (e != cudaSuccess) return fail(c, QTTS_E_CUDA, "qtts_kv8_append: %s", cudaGetErrorString(e));
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
  const int touched = touched_pages(std::min(max_new, n_rows));
  if ((long long)B * touched > 0x7fffffffll) return fail(c, QTTS_E_INVALID, "qtts_kv8_read: too many rows");
  const dim3 grid(B * touched, (2 * f.n_kv_heads + kWarpsPerCta - 1) / kWarpsPerCta);
  const cudaError_t e = launch(f.head_dim == 64 ? read_kernel<64> : read_kernel<128>, grid, kWarpsPerCta * 32,
                               (cudaStream_t)stream, view(c, layer), q, touched, k_out, v_out);
  if (e != cudaSuccess) return fail(c, QTTS_E_CUDA, "qtts_kv8_read: %s", cudaGetErrorString(e));
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
  DeviceGuard g(c->device);
  if (!g.ok) return fail(c, QTTS_E_CUDA, "cudaSetDevice failed");
  const cudaError_t e = kv8_attention(view(c, layer), qb, f.head_dim, f.n_q_heads / f.n_kv_heads, c->G, q, q_stride,
                                      scale, out, out_stride, workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(c, QTTS_E_CUDA, "qtts_kv8_attention: %s", cudaGetErrorString(e));
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
  if (e == cudaSuccess && v) e = cudaMemset(c->dev_err, 0, sizeof(int));
  if (e != cudaSuccess) return fail(c, QTTS_E_CUDA, "qtts_kv8_status: %s", cudaGetErrorString(e));
  if (device_err) *device_err = v;
  if (v == QTTS_DEV_TIMEOUT) return fail(c, QTTS_E_TIMEOUT, "a device-side wait ran out its limit");
  if (v) return fail(c, QTTS_E_DEVICE, "device-side check failed: %d", v);
  return QTTS_OK;
}

}  // extern "C"
