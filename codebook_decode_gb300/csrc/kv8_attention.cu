// kv8_attention.cu -- attention over the 8-bit paged K/V cache.
//
// A tile is up to 8 NT columns (query rows x the q heads of one kv head) of
// one session, against all pages its rows see. Every warp takes whole pages:
//   S^T [16 tokens x columns] = K . Q^T     (A = K codes widened to half)
//   O^T [d x columns]        += V^T . P^T   (A = V codes widened to half)
// on mma.sync m16n8k16 with fp32 accumulators. Tokens stand along the MMA's M,
// so a decode step's few columns fill one n-tile and nothing is padded to 16
// query rows. Codes are exact in half, the blocks' scales are applied outside
// the products: the K scale (with the softmax scale and log2 e) to the fp32
// scores, the V scale to the fp32 weights. Weights are rounded to half
// (2^-12 relative), queries to half after a power of two per column.
//
// Softmax: base 2, per-warp running maximum m of score + log2(V scale), so the
// weights p * s_v that enter the product stay below 2^kSlack whatever the
// scales. m moves only when a value passes m + kSlack (one vote per page, no
// shuffles otherwise). Sums l of the unrounded p in fp32.
//
// The work is counted in units of one page of one kv head, tile after tile. A
// short batch gives each CTA one tile; otherwise the units are cut into equal
// shares, one per CTA, whatever the sessions' lengths. Inside a CTA each warp
// takes an equal run of its units and needs no other warp until all are done:
// a tile that lies inside one warp's run is written from its registers, the
// pieces of others meet in shared memory, and of tiles that several CTAs share
// in the workspace, where the last CTA to arrive joins them in order, so
// results do not depend on which one that is.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace qtts {
namespace {

constexpr int kWaitTries = 1 << 20;  // bound of each wait for a copy (a try suspends for microseconds)
constexpr int kMaxCols = 32;
// A tile of up to this many pages goes to one CTA when there are enough CTAs
// for all tiles: joining pieces through global memory costs more than reading
// the tile with one CTA.
constexpr int kWholePages = 48;

// warps of a CTA, CTAs of an SM, copies in flight per warp (blocks of 32 D bytes)
__host__ __device__ constexpr int warps_of(int NT) { return NT == 1 ? 8 : 4; }
__host__ __device__ constexpr int ctas_of(int NT) { return NT == 1 ? 2 : NT == 2 ? 2 : 1; }
__host__ __device__ constexpr int slots_of(int D, int NT) { return (NT == 4 ? 5 : NT == 2 ? 3 : 2) * (128 / D); }

struct Session {
  int r0, n, L;
};
// dynamic shared memory: copies, each warp's partial of the tile it goes on with
// (its other partial, of a tile that it starts, is its last work and takes its
// copies' place), then per session the units before it and its rows
struct Layout {
  int part, bar, cum, sess, bytes;  // byte offsets
};
__host__ __device__ inline int part_stride(int D) { return D + 4; }  // floats of one column: values, m, l, 2 unused
__host__ __device__ inline Layout layout(int D, int NT, int cols, int B) {
  Layout l;
  const int W = warps_of(NT), S = slots_of(D, NT);
  l.part = W * S * 32 * D;
  l.bar = l.part + W * cols * part_stride(D) * 4;
  l.cum = l.bar + W * S * 8;
  l.sess = l.cum + (B + 1) * 4;
  l.bytes = l.sess + B * (int)sizeof(Session);
  return l;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
// Loads that stay where they are written: before the copies that follow them.
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 load16(const void* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}
template <int KC>
struct RawQuery {
  uint2 q[KC][4];
  float4 cs[4], sn[4];
};
__device__ __forceinline__ bool wait_copy(uint64_t* bar, uint32_t parity) {
  for (int tries = 0; tries < kWaitTries; ++tries)
    if (mbar_test(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
struct Args {
  Kv8View c;
  Kv8Batch q;
  int group, max_cols;
  bool one_each;  // every tile can have its CTA
  const uint16_t* qp;
  int64_t q_stride;
  float scale_log2;
  uint16_t* out;
  int64_t out_stride;
  float* part;        // [2 CTAs][kMaxCols] partial columns
  unsigned* arrived;  // [CTAs] CTAs of the tile that starts in this CTA and ends in a later one; zero between calls
};

// pages that a tile's last row sees
__device__ __forceinline__ int tile_pages(int L, int n) { return (L + n + kPage - 1) / kPage; }

// A part of a tile that one warp worked on: the tile's first unit, pages, first
// packed row, kv head and columns (0: no piece), and whether it reaches its end.
struct Piece {
  int ub, pages, row, h, cols;
  bool ends;
};
// A place in the units: page p of kv head h of session b.
struct Walk {
  int b, h, p, pages;
  Session s;
  const Session* sess;
  int B, nkv;
  __device__ __forceinline__ void enter(int bb) {  // the first session with work from bb on
    for (b = bb; b < B; ++b) {
      s = sess[b];
      if (s.n) break;
    }
    h = p = 0;
    pages = b < B ? tile_pages(s.L, s.n) : 0x7fffffff;
  }
  __device__ __forceinline__ void next_tile() {
    p = 0;
    if (++h == nkv) enter(b + 1);
  }
  __device__ __forceinline__ void advance(int units) {
    p += units;
    while (p >= pages) {
      const int over = p - pages;
      next_tile();
      p = over;
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(warps_of(NT) * 32, ctas_of(NT)) attention_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int W = warps_of(NT), kSlots = slots_of(D, NT);
  constexpr int KC = D / 64;  // 64-dim chunks of a K row
  constexpr int VJ = D / 32;  // 16-byte V words of a lane
  constexpr uint32_t kBytes = 32 * D;
  constexpr int kCol = D + 4;
  const Layout lay = layout(D, NT, a.max_cols, a.q.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem_raw + warp * kSlots * kBytes;
  float* parts = (float*)(smem_raw + lay.part);
  static_assert(8 * NT * kCol * 4 <= kSlots * kBytes, "a partial fits the place of a warp's copies");
  auto piece_col = [&](int i, int col) {  // column of piece i (see s_piece)
    return (i & 1 ? (float*)(smem_raw + (i >> 1) * kSlots * kBytes) : parts + (i >> 1) * a.max_cols * kCol) + col * kCol;
  };
  uint64_t* bars = (uint64_t*)(smem_raw + lay.bar) + warp * kSlots;
  int* cum = (int*)(smem_raw + lay.cum);
  Session* sess = (Session*)(smem_raw + lay.sess);
  __shared__ int s_most, s_pieces[2], s_first[2];
  __shared__ Piece s_piece[2 * W];  // two of each warp: 0 goes on a tile, 1 starts one

  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars[i], 1);
    mbar_init_fence();
    s_piece[2 * warp].cols = s_piece[2 * warp + 1].cols = 0;
  }
  // this CTA's units: [u0, u0 + units) of all; share: units of a CTA, 0: each CTA has one tile
  Walk w;
  w.sess = sess;
  w.B = a.q.B;
  w.nkv = a.c.nkv;
  int u0 = 0, share = 0, units;
  bool whole = a.one_each && a.q.bt_stride <= kWholePages;
  if (!whole) {
    if (warp == 0) {
      int carry = 0, most = 0;
      for (int b0 = 0; b0 < a.q.B; b0 += 32) {
        int x = 0;
        if (b0 + lane < a.q.B) {
          const Kv8Session s = kv8_session(a.q, b0 + lane, a.c.max_context, a.c.err);
          sess[b0 + lane] = {s.r0, s.n, s.L};
          if (s.n) {
            const int p = tile_pages(s.L, s.n);
            most = max(most, p);
            x = p * a.c.nkv;
          }
        }
        const int own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (b0 + lane < a.q.B) cum[b0 + lane] = carry + x - own;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) {
        cum[a.q.B] = carry;
        s_most = most;
      }
    }
    __syncthreads();
    share = (cum[a.q.B] + gridDim.x - 1) / gridDim.x;
    whole = a.one_each && s_most <= max(kWholePages, share + share / 4);
  }
  if (whole) {
    share = 0;
    w.b = blockIdx.x / a.c.nkv;
    if (w.b >= a.q.B) return;
    w.h = blockIdx.x % a.c.nkv;
    const Kv8Session s = kv8_session(a.q, w.b, a.c.max_context, a.c.err);
    if (s.n == 0) return;
    w.s = {s.r0, s.n, s.L};
    w.p = 0;
    units = w.pages = tile_pages(s.L, s.n);
    w.nkv = w.h + 1;  // nothing follows this tile
    w.B = w.b + 1;
  } else {
    // a share below two pages a warp (or a whole short tile) costs more in joining than it saves
    share = max(share, min(s_most, 2 * W));
    const long long at = (long long)blockIdx.x * share;
    const int total = cum[a.q.B];
    if (at >= total) return;
    u0 = (int)at;
    units = min(share, total - u0);
    int lo = 0, hi = a.q.B;  // cum[lo] <= u0 < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= u0) lo = mid;
      else hi = mid;
    }
    w.enter(lo);
    const int per = (cum[lo + 1] - cum[lo]) / a.c.nkv, rem = u0 - cum[lo];
    w.h = rem / per;
    w.p = rem - w.h * per;
  }
  // this warp's units, as offsets from u0
  const int n0 = (int)((long long)units * warp / W), n1 = (int)((long long)units * (warp + 1) / W);
  const int count = n1 - n0;
  w.advance(n0);

  // lane x holds the block and scales of this warp's unit 32 k + x; those of
  // the next 32 are fetched meanwhile
  Walk wf = w;
  auto fetch_block = [&](int k) {
    int blk = 0;
    if (32 * k < count) {
      Walk x = wf;
      if (32 * k + lane < count) {
        x.advance(lane);
        int page = a.q.bt[(size_t)x.b * a.q.bt_stride + x.p];
        if (page < 0 || page >= a.c.pool_pages) {
          set_err(a.c.err, QTTS_DEV_BAD_PAGE);
          page = 0;  // inside the pool; the session's result is not used
        }
        blk = page * a.c.nkv + x.h;
      }
      if (32 * (k + 1) < count) wf.advance(32);
    }
    return blk;
  };
  auto fetch_scale = [&](int b) {
    const uint2 v = load8(a.c.scales + 2 * (size_t)b);
    return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  };
  // a column's query and its rotation, as they stand in memory
  auto load_q = [&](RawQuery<KC>& r, int nt) {
    const int col = nt * 8 + g, qr = col / a.group, cols = w.s.n * a.group;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) r.q[c][e] = make_uint2(0u, 0u);
    if (col < cols) {
      const uint16_t* src = a.qp + (int64_t)(w.s.r0 + qr) * a.q_stride +
                            (size_t)(w.h * a.group + col - qr * a.group) * D + 16 * t4;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) r.q[c][e] = load8(src + 64 * c + 4 * e);
    }
    if (a.c.rope_cos) {
      const size_t at = (size_t)(w.s.L + min(qr, w.s.n - 1)) * (D / 2) + 16 * (D == 128 ? t4 : t4 & 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r.cs[e] = load16(a.c.rope_cos + at + 4 * e);
        r.sn[e] = load16(a.c.rope_sin + at + 4 * e);
      }
    }
  };

  // The first tile's queries are asked for before the first copies: behind them
  // they would wait for every SM's copies in the memory queues.
  RawQuery<KC> raw;
  if (NT == 1 && count) load_q(raw, 0);
  int blk = fetch_block(0), blk_next = 0;
  float2 scl = fetch_scale(blk), scl_next = make_float2(0.f, 0.f);
  int n = 0;  // units done: slot n % kSlots, parity n / kSlots
  bool dead = false;
  auto issue = [&](int k) {  // copy the block of unit k, at most kSlots ahead of n
    const int from = __shfl_sync(0xffffffffu, (k ^ n) & 32 ? blk_next : blk, k & 31);
    if (lane == 0 && !dead && k < count) {
      uint64_t* bar = &bars[k % kSlots];
      mbar_arrive_expect_tx(bar, kBytes);
      bulk_load(ring + k % kSlots * kBytes, a.c.codes + (size_t)from * kBytes, kBytes, bar);
    }
  };
#pragma unroll
  for (int k = 0; k < kSlots; ++k) issue(k);

  auto write = [&](int row, int h, int col, int at, float4 v, float sum) {
    const int qr = col / a.group;
    uint16_t* dst = a.out + (int64_t)(row + qr) * a.out_stride + (size_t)(h * a.group + col - qr * a.group) * D + at;
    const float r = 1.f / sum;
    *(uint2*)dst = make_uint2(f2bf(v.x * r) | (uint32_t)f2bf(v.y * r) << 16,
                              f2bf(v.z * r) | (uint32_t)f2bf(v.w * r) << 16);
  };

  while (n < count) {
    const int seg_end = min(count, n + w.pages - w.p);
    const int seg0 = n, p0 = w.p;
    const int cols = w.s.n * a.group;
    // queries: rotated, scaled by a power of two per column, as B fragments
    uint32_t qf[NT][KC * 4][2];
    float cf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1 || n > 0) load_q(raw, nt);
      float x[KC][16];
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[c][4 * e] = bf2f(raw.q[c][e].x & 0xffffu);
          x[c][4 * e + 1] = __uint_as_float(raw.q[c][e].x & 0xffff0000u);
          x[c][4 * e + 2] = bf2f(raw.q[c][e].y & 0xffffu);
          x[c][4 * e + 3] = __uint_as_float(raw.q[c][e].y & 0xffff0000u);
        }
      if (a.c.rope_cos) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float* cs = &raw.cs[e / 4].x;
          const float* sn = &raw.sn[e / 4].x;
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            if constexpr (D == 128) {
              const float u = x[0][e + f], v = x[1][e + f];
              x[0][e + f] = u * cs[f] - v * sn[f];
              x[1][e + f] = v * cs[f] + u * sn[f];
            } else {  // the partner dim stands two lanes further
              const float u = x[0][e + f], v = __shfl_xor_sync(0xffffffffu, u, 2);
              x[0][e + f] = t4 < 2 ? u * cs[f] - v * sn[f] : u * cs[f] + v * sn[f];
            }
          }
        }
      }
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = max(mx, __float_as_uint(x[c][e]) & 0x7f800000u);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^e of the largest magnitude, kept where its reciprocal is a normal number
      const uint32_t ex = min(max(mx, 1u << 23), 253u << 23);
      const float inv = __uint_as_float((254u << 23) - ex);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qf[nt][c * 4 + e][0] = half2_bits(x[c][4 * e] * inv, x[c][4 * e + 1] * inv);
          qf[nt][c * 4 + e][1] = half2_bits(x[c][4 * e + 2] * inv, x[c][4 * e + 3] * inv);
        }
      const float f = __uint_as_float(ex) * a.scale_log2;
      cf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);  // columns 2 t4 and 2 t4 + 1
      cf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
    }
    // last token that this lane's columns see
    int see[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) see[nt][e] = w.s.L + min((nt * 8 + 2 * t4 + e) / a.group, w.s.n - 1);
    const int first_masked = (w.s.L + 1) / kPage;  // pages before this one are seen whole by every row

    float o[NT][VJ * 2][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < VJ * 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
    }
    for (; n < seg_end; ++n) {
      if ((n & 31) == 0) {
        if (n) {
          blk = blk_next;
          scl = scl_next;
        }
        blk_next = fetch_block((n >> 5) + 1);
      } else if ((n & 31) == 16) {
        scl_next = fetch_scale(blk_next);
      }
      const int slot = n % kSlots;
      if (!dead && !__all_sync(0xffffffffu, wait_copy(&bars[slot], (n / kSlots) & 1))) {
        // no more copies; those in flight get one more wait, so that none lands after the CTA has left
        dead = true;
        set_err(a.c.err, QTTS_DEV_TIMEOUT);
        for (int k = n; k < min(n + kSlots, count); ++k) wait_copy(&bars[k % kSlots], (k / kSlots) & 1);
      }
      const uint8_t* kb = ring + slot * kBytes;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 ka = *(const uint4*)(kb + c * 1024 + g * 64 + t4 * 16);
        const uint4 kc = *(const uint4*)(kb + c * 1024 + (g + 8) * 64 + t4 * 16);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a0, a1, a2, a3;
          widen(wa[e], a0, a2);
          widen(wc[e], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[nt], a0, a1, a2, a3, qf[nt][c * 4 + e][0], qf[nt][c * 4 + e][1]);
        }
      }
      uint4 vw[VJ];
#pragma unroll
      for (int j = 0; j < VJ; ++j) vw[j] = *(const uint4*)(kb + 16 * D + (8 * j + g) * 64 + t4 * 16);
      __syncwarp();
      issue(n + kSlots);

      const float2 sc = make_float2(__shfl_sync(0xffffffffu, scl.x, n & 31), __shfl_sync(0xffffffffu, scl.y, n & 31));
      const float lv = lg2(fmaxf(sc.y, kKv8MinScale)) + (sc.y != sc.y ? sc.y : 0.f);
      const int page = p0 + n - seg0;
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = sc.x * cf[nt][e];
          s[nt][e] *= f;
          s[nt][e + 2] *= f;
          if (page >= first_masked) {
            if (page * kPage + g > see[nt][e]) s[nt][e] = -INFINITY;
            if (page * kPage + g + 8 > see[nt][e]) s[nt][e + 2] = -INFINITY;
          }
          grow |= fmaxf(s[nt][e], s[nt][e + 2]) + lv > m[nt][e] + kSlack;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[nt][e], s[nt][e + 2]) + lv;
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            mx = fmaxf(mx, m[nt][e]);
            const float f = ex2(m[nt][e] - mx);
            m[nt][e] = mx;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < VJ * 2; ++j) {
              o[nt][j][e] *= f;
              o[nt][j][e + 2] *= f;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2(s[nt][e] - m[nt][e & 1]);
        l[nt][0] += p[0] + p[2];
        l[nt][1] += p[1] + p[3];
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p[e] * sc.y;
        if (page >= first_masked) {  // what a column does not see gives nothing, whatever its scale
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = p[e] > 0.f || p[e] != p[e] ? v[e] : 0.f;
        }
        pf[nt][0] = transpose8(half2_bits(v[0], v[1]));
        pf[nt][1] = transpose8(half2_bits(v[2], v[3]));
      }
#pragma unroll
      for (int j = 0; j < VJ; ++j) {
        const uint32_t w[4] = {vw[j].x, vw[j].y, vw[j].z, vw[j].w};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t a0, a1, a2, a3;
          widen(w[2 * p], a0, a2);
          widen(w[2 * p + 1], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * j + p], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        }
      }
    }

    // sums over the lanes of a column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], k);
    const bool starts = p0 == 0, ends = p0 + seg_end - seg0 == w.pages;
    float* dst = piece_col(2 * warp + starts, 0);
    __syncwarp();  // the last copies have been read
    if (!(starts && ends) && lane == 0)
      s_piece[2 * warp + starts] = {u0 + n0 + seg0 - p0, w.pages, w.s.r0, w.h, cols, ends};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = nt * 8 + 2 * t4 + e;
        if (col < cols) {
#pragma unroll
          for (int j = 0; j < VJ; ++j) {
            const float4 v = make_float4(o[nt][2 * j][e], o[nt][2 * j][e + 2], o[nt][2 * j + 1][e], o[nt][2 * j + 1][e + 2]);
            if (starts && ends) write(w.s.r0, w.h, col, 32 * j + 4 * g, v, l[nt][e]);
            else *(float4*)(dst + col * kCol + 32 * j + 4 * g) = v;
          }
          if (!(starts && ends) && g == 0) *(float2*)(dst + col * kCol + D) = make_float2(m[nt][e], l[nt][e]);
        }
      }
    w.p += seg_end - seg0;
    if (ends) w.next_tile();
  }

  __syncthreads();
  // Pieces of one tile stand in warp order: first the one that starts it (odd),
  // then those that go on (even). Each run of them is joined by the warps, one
  // column at a time. Runs that began in an earlier CTA or go on in a later one
  // leave a partial: a CTA starts at most one shared tile (1) and goes on with
  // at most one (0).
  uint32_t valid = __ballot_sync(0xffffffffu, lane < 2 * W && s_piece[lane % (2 * W)].cols);
  const uint32_t ended = __ballot_sync(0xffffffffu, lane < 2 * W && s_piece[lane % (2 * W)].ends) & valid;
  int open0 = -1, open1 = -1, item = 0;  // first piece of each shared run
  while (valid) {
    const int from = __ffs(valid) - 1;
    const uint32_t e = ended & (~0u << from), upto = e ? (e ^ (e - 1)) : ~0u, run = valid & upto;
    valid &= ~upto;
    const bool closed = (from & 1) && e;
    if (!closed) (from & 1 ? open1 : open0) = from;
    const Piece& pc = s_piece[from];
    for (int col = 0; col < pc.cols; ++col) {
      if (item++ % W != warp) continue;
      const bool in = run >> lane & 1;
      const float2 ml = in ? *(const float2*)(piece_col(lane, col) + D) : make_float2(kNone, 0.f);
      const float mx = warp_max(ml.x), f = ex2(ml.x - mx), sum = warp_sum(ml.y * f);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t k = run; k; k &= k - 1) {
        const int i = __ffs(k) - 1;
        const float fi = __shfl_sync(0xffffffffu, f, i);
        if (lane < D / 4) axpy(v, *(const float4*)(piece_col(i, col) + 4 * lane), fi);
      }
      if (closed) {
        if (lane < D / 4) write(pc.row, pc.h, col, 4 * lane, v, sum);
      } else {
        float* dst = a.part + ((size_t)(2 * blockIdx.x + (from & 1)) * kMaxCols + col) * kCol;
        if (lane < D / 4) *(float4*)(dst + 4 * lane) = v;
        if (lane == 0) *(float2*)(dst + D) = make_float2(mx, sum);
      }
    }
  }
  if (open0 < 0 && open1 < 0) return;
  __threadfence();
  __syncthreads();
  const int mine = tid == 0 ? open0 : open1;
  if (tid < 2 && mine >= 0) {
    const Piece& pc = s_piece[mine];
    const int c0 = pc.ub / share, pieces = (pc.ub + pc.pages - 1) / share - c0 + 1;
    s_pieces[tid] = atomicAdd(&a.arrived[c0], 1u) == (unsigned)pieces - 1 ? pieces : 0;
    s_first[tid] = c0;
  }
  __syncthreads();
  for (int which = 0; which < 2; ++which) {
    const int from = which ? open1 : open0, pieces = from >= 0 ? s_pieces[which] : 0, c0 = s_first[which];
    if (!pieces) continue;
    __threadfence();
    const Piece pc = s_piece[from];
    // few columns: several warps share one, each with every `per`-th partial
    const int per = pc.cols >= W ? 1 : pc.cols > W / 2 ? 1 : pc.cols > W / 4 ? 2 : pc.cols > W / 8 ? 4 : W;
    const int gi = warp % per;
    for (int col = warp / per; col < pc.cols; col += W / per) {
      float mx = kNone, sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      auto partial = [&](int i) {
        return a.part + ((size_t)(2 * (c0 + i) + (i == 0)) * kMaxCols + col) * kCol;
      };
      for (int i0 = gi; i0 < pieces; i0 += 32 * per) {
        const int i = i0 + lane * per;
        const float2 ml = i < pieces ? __ldcg((const float2*)(partial(i) + D)) : make_float2(kNone, 0.f);
        const float nm = fmaxf(mx, warp_max(ml.x)), f0 = ex2(mx - nm), f1 = ex2(ml.x - nm);
        mx = nm;
        sum = sum * f0 + warp_sum(ml.y * f1);
        v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
        for (int k = 0; k < 32 && i0 + k * per < pieces; k += 8) {
          float4 y[8];  // eight loads in flight
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int ik = i0 + (k + e) * per;
            y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < D / 4 && ik < pieces) y[e] = __ldcg((const float4*)(partial(ik) + 4 * lane));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) axpy(v, y[e], __shfl_sync(0xffffffffu, f1, k + e));
        }
      }
      if (per == 1) {
        if (lane < D / 4) write(pc.row, pc.h, col, 4 * lane, v, sum);
      } else {
        float* dst = parts + warp * kCol;
        if (lane < D / 4) *(float4*)(dst + 4 * lane) = v;
        if (lane == 0) *(float2*)(dst + D) = make_float2(mx, sum);
      }
    }
    if (per > 1) {
      __syncthreads();
      if (gi == 0 && warp / per < pc.cols) {
        float mx = kNone, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < per; ++k) mx = fmaxf(mx, parts[(warp + k) * kCol + D]);
        for (int k = 0; k < per; ++k) {
          const float* src = parts + (warp + k) * kCol;
          const float f = ex2(src[D] - mx);
          sum += src[D + 1] * f;
          if (lane < D / 4) axpy(v, *(const float4*)(src + 4 * lane), f);
        }
        if (lane < D / 4) write(pc.row, pc.h, warp / per, 4 * lane, v, sum);
      }
      __syncthreads();
    }
    if (tid == 0) a.arrived[c0] = 0;  // ready for the next call
  }
}

template <int D, int NT>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              layout(D, NT, 8 * NT, kKv8MaxBatch).bytes);
}
template <int D, int NT>
cudaError_t launch_one(const Args& a, int sms, cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(a.one_each && a.q.bt_stride <= kWholePages ? a.q.B * a.c.nkv : sms * ctas_of(NT));
  lc.blockDim = dim3(32 * warps_of(NT));
  lc.dynamicSmemBytes = layout(D, NT, a.max_cols, a.q.B).bytes;
  lc.stream = s;
  return cudaLaunchKernelEx(&lc, attention_kernel<D, NT>, a);
}

}  // namespace

cudaError_t kv8_attention_setup(int d) {
  cudaError_t e = kv8_chunk_setup(d);
  if (e != cudaSuccess) return e;
  if (d == 64) {
    (e = setup_one<64, 1>()) || (e = setup_one<64, 2>()) || (e = setup_one<64, 4>());
  } else {
    (e = setup_one<128, 1>()) || (e = setup_one<128, 2>()) || (e = setup_one<128, 4>());
  }
  return e;
}

// the arrival counts, then two partial tiles for each CTA of the largest grid
size_t kv8_attention_workspace(int d, int sms) {
  const size_t ctas = 2 * (size_t)sms;
  return ctas * sizeof(unsigned) + std::max(2 * ctas * kMaxCols * (d + 4) * sizeof(float), kv8_chunk_workspace(d, sms));
}

cudaError_t kv8_attention(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                          int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, void* work, cudaStream_t s) {
  // places in the units are 32-bit
  const long long tiles = (q.max_new + 0ll) * group / 8 + 1, pages = std::min(q.bt_stride, v.max_context / kPage + 1);
  if (q.B * pages * v.nkv >= (1ll << 31) / std::max(tiles, 1ll)) return cudaErrorInvalidValue;
  // the fewest n-tiles that hold every session's columns; more rows go in tiles of 32 columns
  const long long cols = (long long)q.max_new * group;
  float* part = (float*)((char*)work + 2 * (size_t)sms * sizeof(unsigned));
  if (cols > kMaxCols)
    return kv8_chunk(v, q, d, group, sms, qp, q_stride, scale, out, out_stride, (unsigned*)work, part, s);
  const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
  Args a{};
  a.c = v;
  a.q = q;
  a.group = group;
  a.max_cols = (int)cols;
  a.one_each = (long long)q.B * v.nkv <= sms * ctas_of(nt);
  a.qp = qp;
  a.q_stride = q_stride;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.out_stride = out_stride;
  a.arrived = (unsigned*)work;
  a.part = part;
  if (d == 64)
    return nt == 1 ? launch_one<64, 1>(a, sms, s) : nt == 2 ? launch_one<64, 2>(a, sms, s) : launch_one<64, 4>(a, sms, s);
  return nt == 1 ? launch_one<128, 1>(a, sms, s) : nt == 2 ? launch_one<128, 2>(a, sms, s) : launch_one<128, 4>(a, sms, s);
}

}  // namespace qtts
