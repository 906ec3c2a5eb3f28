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
// (2^-11 relative), queries to half after a power of two per column.
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
//
// Bound by bytes for long sessions (one token each of 32 sessions of 4000 to 16000,
// 16 q and 8 kv heads of 128: 108 us, 6.1 TB/s; one of 130000: 49 us, 5.4 TB/s), by
// the chain of lengths, table, copies, softmax and join for short ones (8 sessions of
// 64 to 512: 8 us; from tables of 16384 pages, where the tiles have to be counted first, 9).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace qtts {
namespace {

constexpr int kWaitTries = 1 << 20;  // bound of each wait for a copy (a try suspends for microseconds)
// Columns of a tile, at most; calls with more go to the tcgen05 kernel. Measured on both
// sides: 32 columns (16 rows, 2 q heads a kv head) behind 100 tokens 16.8 us here, 9.1
// there, 32 sessions of them behind 8000 295 and 220; 16 columns 8.5 (8 sessions, 100
// tokens) and 9.4, 110 (32 sessions, 8000) and 219.
constexpr int kMaxCols = 16;
// A tile of up to kWholePages pages goes to one CTA when there are enough CTAs
// for all tiles, up to kWholePagesMany when the tiles take half of the CTAs:
// joining pieces through global memory costs more than reading the tile with
// one CTA (32 sessions of 100..1200 tokens: 21.8 us cut, 18.1 whole).
constexpr int kWholePages = 48, kWholePagesMany = 96;
constexpr int kTiles = 8;  // tiles whose queries a CTA prepares at a time, at most

// warps of a CTA, CTAs of an SM, copies in flight per warp (blocks of 32 D bytes)
__host__ __device__ constexpr int warps_of(int NT) { return NT == 1 ? 8 : 4; }
constexpr int kCtas = 2;
__host__ __device__ constexpr int slots_of(int D, int NT) { return (NT == 2 ? 3 : 2) * (128 / D); }

struct Session {
  int r0, n, L;
};
// dynamic shared memory: copies, each warp's partial of the tile it goes on with
// (its other partial, of a tile that it starts, is its last work and takes its
// copies' place), the tiles' queries, then per session the units before it and
// its rows
struct Layout {
  int part, bar, query, cum, sess, tiles, bytes;  // byte offsets; tiles: queries prepared at a time
};
__host__ __device__ constexpr int query_stride(int D) { return 2 * D + 16; }  // bytes of a column: rows of a load on different banks
__host__ __device__ inline Layout layout(int D, int NT, int cols, int B) {
  Layout l;
  const int W = warps_of(NT), S = slots_of(D, NT);
  l.tiles = cols <= 4 ? kTiles : 4;
  l.part = W * S * 32 * D;
  l.bar = l.part + W * cols * (D + 4) * 4;  // floats of one column: values, maximum, sum, 2 unused
  l.query = l.bar + W * S * 8;
  l.cum = l.query + l.tiles * cols * query_stride(D);
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
// A tile (or the part of it) that a CTA works on: `units` pages from page0 on,
// the first of them at unit `off` of the CTA's present tiles.
struct Tile {
  int b, h, r0, n, L, pages, page0, off, units, ub;
};

template <int D, int NT>
__global__ void __launch_bounds__(warps_of(NT) * 32, kCtas) attention_kernel(const __grid_constant__ Args a) {
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
  uint8_t* queries = smem_raw + lay.query;
  int* cum = (int*)(smem_raw + lay.cum);
  Session* sess = (Session*)(smem_raw + lay.sess);
  __shared__ int s_units, s_share, s_pieces[2], s_first[2], s_tiles, s_sub;
  __shared__ Piece s_piece[2 * W];  // two of each warp: 0 goes on a tile, 1 starts one
  __shared__ Tile s_tile[kTiles];
  __shared__ float s_cf[kTiles][8 * NT];

  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&bars[i], 1);
    mbar_init_fence();
  }
  grid_dependency_wait();

  // warp 0: this CTA's units [u0, u0 + units) of all, the tile that they begin in
  // and the page in it; share: units of a CTA, 0: each CTA has one tile
  int u0 = 0, units = 0, share = 0, b = 0, h = 0, page = 0;
  if (warp == 0) {
    bool whole = a.one_each && a.q.bt_stride <= kWholePages;
    int carry = 0, most = 0;
    for (int b0 = 0; b0 < a.q.B && !whole; b0 += 32) {
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
    if (!whole) {
      if (lane == 0) cum[a.q.B] = carry;
      __syncwarp();
      most = __reduce_max_sync(0xffffffffu, most);
      share = (carry + gridDim.x - 1) / gridDim.x;
      whole = a.one_each && most <= max(2 * a.q.B * a.c.nkv >= gridDim.x ? kWholePagesMany : kWholePages, share + share / 4);
    }
    if (whole) {
      share = 0;
      b = blockIdx.x / a.c.nkv;
      h = blockIdx.x % a.c.nkv;
      if (b < a.q.B) {
        const Kv8Session s = kv8_session(a.q, b, a.c.max_context, a.c.err);
        if (s.n) units = tile_pages(s.L, s.n);
        if (lane == 0) sess[b] = {s.r0, s.n, s.L};
        __syncwarp();
      }
    } else {
      // a share below two pages a warp (or a whole short tile) costs more in joining than it saves
      share = max(share, min(most, 2 * W));
      const long long at = (long long)blockIdx.x * share;
      if (at < carry) {
        u0 = (int)at;
        units = min(share, carry - u0);
        int hi = a.q.B;  // cum[b] <= u0 < cum[hi]
        while (hi - b > 1) {
          const int mid = (b + hi) >> 1;
          if (cum[mid] <= u0) b = mid;
          else hi = mid;
        }
        const int per = (cum[b + 1] - cum[b]) / a.c.nkv, rem = u0 - cum[b];
        h = rem / per;
        page = rem - h * per;
      }
    }
    if (lane == 0) {
      s_units = units;
      s_share = share;
    }
  }

  // the next tiles of this CTA (warp 0 keeps the place), up to the layout's number
  auto next_tiles = [&]() {
    if (warp == 0) {
      int t = 0, off = 0;
      while (t < lay.tiles && units > 0) {
        const Session s = sess[b];
        if (s.n) {
          Tile x{b, h, s.r0, s.n, s.L, tile_pages(s.L, s.n), page, off, 0, u0 + off - page};
          x.units = min(x.pages - page, units);
          if (lane == 0) s_tile[t] = x;
          off += x.units;
          units -= x.units;
          page = 0;
          ++t;
        }
        if (s.n == 0 || ++h == a.c.nkv) {
          h = 0;
          ++b;
        }
      }
      u0 += off;
      if (lane == 0) {
        s_tiles = t;
        s_sub = off;
      }
    }
    if (tid < 2 * W) s_piece[tid].cols = 0;
    __syncthreads();
  };
  next_tiles();
  const int cta_units = s_units;
  share = s_share;
  bool dead = false;
  auto write = [&](int row, int h, int col, int at, float4 v, float sum) {
    const int qr = col / a.group;
    uint16_t* dst = a.out + (int64_t)(row + qr) * a.out_stride + (size_t)(h * a.group + col - qr * a.group) * D + at;
    const float r = 1.f / sum;
    *(uint2*)dst = make_uint2(f2bf(v.x * r) | (uint32_t)f2bf(v.y * r) << 16,
                              f2bf(v.z * r) | (uint32_t)f2bf(v.w * r) << 16);
  };

  int slot = 0, parity = 0;  // of this warp's next copy
  for (int done = 0; done < cta_units;) {
    const int sub = s_sub, ntiles = s_tiles;
    // this warp's units of the present tiles
    const int n0 = (int)((long long)sub * warp / W), count = (int)((long long)sub * (warp + 1) / W) - n0;

    // lane x holds the block and scales of this warp's unit 32 k + x; those of
    // the next 32 are fetched meanwhile
    auto fetch_block = [&](int k) {
      const int unit = n0 + 32 * k + lane;
      if (32 * k + lane >= count) return 0;
      int t = 0;
      while (t + 1 < ntiles && s_tile[t + 1].off <= unit) ++t;
      int pg = a.q.bt[(size_t)s_tile[t].b * a.q.bt_stride + s_tile[t].page0 + unit - s_tile[t].off];
      if (pg < 0 || pg >= a.c.pool_pages) {
        set_err(a.c.err, QTTS_DEV_BAD_PAGE);
        pg = 0;  // inside the pool; the session's result is not used
      }
      return pg * a.c.nkv + s_tile[t].h;
    };
    auto fetch_scale = [&](int id) { return *(const float2*)(a.c.scales + 2 * (size_t)id); };

    // The tiles' queries: rotated, scaled by a power of two per column, as half.
    // A thread takes 4 dims of a column and their rotation partners D/2 further.
    // They are asked for before the first copies: behind them they would wait
    // for every SM's copies in the memory queues.
    constexpr int kQuads = D / 8;
    struct Item {
      uint2 lo, hi;
      float4 cs, sn;
    } it;
    const int items = ntiles * a.max_cols * kQuads;
    auto load_item = [&](int i) {
      it.lo = it.hi = make_uint2(0u, 0u);
      it.cs = make_float4(1.f, 1.f, 1.f, 1.f);
      it.sn = make_float4(0.f, 0.f, 0.f, 0.f);
      const int r = i / kQuads, t = r / a.max_cols, col = r - t * a.max_cols, at = i % kQuads * 4;
      if (i < items && col < s_tile[t].n * a.group) {
        const int qr = col / a.group;
        const uint16_t* src = a.qp + (int64_t)(s_tile[t].r0 + qr) * a.q_stride +
                              (size_t)(s_tile[t].h * a.group + col - qr * a.group) * D + at;
        it.lo = load8(src);
        it.hi = load8(src + D / 2);
        if (a.c.rope_cos) {
          const size_t row = (size_t)(s_tile[t].L + qr) * (D / 2) + at;
          it.cs = load16(a.c.rope_cos + row);
          it.sn = load16(a.c.rope_sin + row);
        }
      }
    };
    auto put_item = [&](int i) {
      // power of two of the column's largest magnitude (before the rotation, which
      // can grow it by sqrt 2: half has room), kept where its reciprocal is normal
      uint32_t mag = __vmaxu2(__vmaxu2(it.lo.x & 0x7fff7fffu, it.lo.y & 0x7fff7fffu),
                              __vmaxu2(it.hi.x & 0x7fff7fffu, it.hi.y & 0x7fff7fffu));
      mag = max(mag & 0xffffu, mag >> 16);
#pragma unroll
      for (int o = 1; o < kQuads; o <<= 1) mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
      const uint32_t ex = min(max(mag << 16 & 0x7f800000u, 1u << 23), 253u << 23);
      const float inv = __uint_as_float((254u << 23) - ex);
      const float lo[4] = {bf2f(it.lo.x & 0xffffu), __uint_as_float(it.lo.x & 0xffff0000u), bf2f(it.lo.y & 0xffffu),
                           __uint_as_float(it.lo.y & 0xffff0000u)};
      const float hi[4] = {bf2f(it.hi.x & 0xffffu), __uint_as_float(it.hi.x & 0xffff0000u), bf2f(it.hi.y & 0xffffu),
                           __uint_as_float(it.hi.y & 0xffff0000u)};
      const float cs[4] = {it.cs.x, it.cs.y, it.cs.z, it.cs.w}, sn[4] = {it.sn.x, it.sn.y, it.sn.z, it.sn.w};
      float u[4], v[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const float p = lo[f] * inv, q = hi[f] * inv;
        u[f] = p;
        v[f] = q;
        if (a.c.rope_cos) {
          u[f] = p * cs[f] - q * sn[f];
          v[f] = q * cs[f] + p * sn[f];
        }
      }
      if (i < items) {
        const int r = i / kQuads;
        uint8_t* dst = queries + r * query_stride(D) + i % kQuads * 8;
        *(uint2*)dst = make_uint2(half2_bits(u[0], u[1]), half2_bits(u[2], u[3]));
        *(uint2*)(dst + D) = make_uint2(half2_bits(v[0], v[1]), half2_bits(v[2], v[3]));
        if (i % kQuads == 0) s_cf[r / a.max_cols][r % a.max_cols] = __uint_as_float(ex) * a.scale_log2;
      }
    };

    load_item(tid);
    int blk = fetch_block(0), blk_next = 0;
    float2 scl = fetch_scale(blk), scl_next = make_float2(0.f, 0.f);
    int n = 0;  // units done
    auto issue = [&](int k, int to) {  // copy the block of unit k, at most kSlots ahead of n
      const int from = __shfl_sync(0xffffffffu, (k ^ n) & 32 ? blk_next : blk, k & 31);
      if (lane == 0 && !dead && k < count) {
        mbar_arrive_expect_tx(&bars[to], kBytes);
        bulk_load(ring + to * kBytes, a.c.codes + (size_t)from * kBytes, kBytes, &bars[to]);
      }
    };
    if (done) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // partials stood where copies go now
#pragma unroll
    for (int k = 0; k < kSlots; ++k) issue(k, slot + k < kSlots ? slot + k : slot + k - kSlots);
    for (int i0 = warp * 32; i0 < items; i0 += W * 32) {
      put_item(i0 + lane);
      if (i0 + W * 32 < items) load_item(i0 + W * 32 + lane);
    }
    __syncthreads();

    int j = 0;  // the tile at hand
    while (j + 1 < ntiles && s_tile[j + 1].off <= n0) ++j;
    while (n < count) {
      const Tile& T = s_tile[j];
      const int seg_end = min(count, T.off + T.units - n0), seg0 = n, p0 = T.page0 + n0 + n - T.off;
      const int cols = T.n * a.group;
      // queries as B fragments
      uint32_t qf[NT][KC * 4][2];
      float cf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint8_t* src = queries + (j * a.max_cols + min(nt * 8 + g, cols - 1)) * query_stride(D) + 32 * t4;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 q4 = *(const uint4*)(src + 128 * c + 16 * e);
            qf[nt][c * 4 + 2 * e][0] = q4.x;
            qf[nt][c * 4 + 2 * e][1] = q4.y;
            qf[nt][c * 4 + 2 * e + 1][0] = q4.z;
            qf[nt][c * 4 + 2 * e + 1][1] = q4.w;
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) cf[nt][e] = s_cf[j][min(nt * 8 + 2 * t4 + e, cols - 1)];
      }
      // last token that this lane's columns see
      int see[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) see[nt][e] = T.L + min((nt * 8 + 2 * t4 + e) / a.group, T.n - 1);
      const int first_masked = (T.L + 1) / kPage;  // pages before this one are seen whole by every row

      float o[NT][VJ * 2][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = kNone;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < VJ * 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
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
        if (!dead && !__all_sync(0xffffffffu, wait_copy(&bars[slot], parity))) {
          // no more copies; those in flight get one more wait, so that none lands after the CTA has left
          dead = true;
          set_err(a.c.err, QTTS_DEV_TIMEOUT);
          for (int k = 0, s = slot, p = parity; k < kSlots && n + k < count; ++k) {
            wait_copy(&bars[s], p);
            if (++s == kSlots) {
              s = 0;
              p ^= 1;
            }
          }
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
        issue(n + kSlots, slot);

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
              l[nt][e] = rebase(l[nt][e], m[nt][e], mx);
              m[nt][e] = mx;
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
            for (int e = 0; e < 4; ++e) v[e] = page * kPage + g + (e >> 1) * 8 > see[nt][e & 1] ? 0.f : v[e];
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
        if (++slot == kSlots) {
          slot = 0;
          parity ^= 1;
        }
      }

      // sums over the lanes of a column
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], k);
      const bool starts = p0 == 0, ends = p0 + seg_end - seg0 == T.pages;
      float* dst = piece_col(2 * warp + starts, 0);
      __syncwarp();  // the last copies have been read
      if (!(starts && ends) && lane == 0) s_piece[2 * warp + starts] = {T.ub, T.pages, T.r0, T.h, cols, ends};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = nt * 8 + 2 * t4 + e;
          if (col < cols) {
#pragma unroll
            for (int i = 0; i < VJ; ++i) {
              const float4 v = make_float4(o[nt][2 * i][e], o[nt][2 * i][e + 2], o[nt][2 * i + 1][e], o[nt][2 * i + 1][e + 2]);
              if (starts && ends) write(T.r0, T.h, col, 32 * i + 4 * g, v, l[nt][e]);
              else *(float4*)(dst + col * kCol + 32 * i + 4 * g) = v;
            }
            if (!(starts && ends) && g == 0) *(float2*)(dst + col * kCol + D) = make_float2(m[nt][e], l[nt][e]);
          }
        }
      if (n0 + seg_end == T.off + T.units) ++j;
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
        const float mx = warp_max(ml.x), f = ex2(ml.x - mx), sum = warp_sum(rebase(ml.y, ml.x, mx));
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
    const bool shared = open0 >= 0 || open1 >= 0;
    if (shared) __threadfence();
    if (shared) __syncthreads();
    const int mine = tid == 0 ? open0 : open1;
    if (shared && tid < 2 && mine >= 0) {
      const Piece& pc = s_piece[mine];
      const int c0 = pc.ub / share, pieces = (pc.ub + pc.pages - 1) / share - c0 + 1;
      s_pieces[tid] = atomicAdd(&a.arrived[c0], 1u) == (unsigned)pieces - 1 ? pieces : 0;
      s_first[tid] = c0;
    }
    if (shared) __syncthreads();
    for (int which = 0; which < 2 && shared; ++which) {
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
          sum = rebase(sum, mx, nm) + warp_sum(rebase(ml.y, ml.x, nm));
          mx = nm;
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
            sum += rebase(src[D + 1], src[D], mx);
            if (lane < D / 4) axpy(v, *(const float4*)(src + 4 * lane), f);
          }
          if (lane < D / 4) write(pc.row, pc.h, warp / per, 4 * lane, v, sum);
        }
        __syncthreads();
      }
      if (tid == 0) a.arrived[c0] = 0;  // ready for the next call
    }

    done += sub;
    if (done < cta_units) {
      __syncthreads();
      next_tiles();
    }
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
  cudaLaunchAttribute at[1];
  early_launch(lc, at);
  lc.gridDim = dim3(a.one_each && a.q.bt_stride <= kWholePages ? a.q.B * a.c.nkv : sms * kCtas);
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
    (e = setup_one<64, 1>()) || (e = setup_one<64, 2>());
  } else {
    (e = setup_one<128, 1>()) || (e = setup_one<128, 2>());
  }
  return e;
}

// the arrival counts, then two partial tiles for each CTA of the largest grid
size_t kv8_attention_workspace(int d, int sms) {
  const size_t ctas = kCtas * (size_t)sms;
  return ctas * sizeof(unsigned) + std::max(2 * ctas * kMaxCols * (d + 4) * sizeof(float), kv8_chunk_workspace(d, sms));
}

// pages of a session, at most
static long long most_pages(const Kv8View& v, const Kv8Batch& q) {
  return std::min((long long)q.bt_stride, v.max_context / kPage + 1ll);
}

// Places in the work are 32-bit: pages of all sessions and kv heads, or key
// steps of all tiles. What a call can need at most, from its sizes.
bool kv8_attention_fits(const Kv8View& v, const Kv8Batch& q, int group) {
  const long long pages = most_pages(v, q);
  return q.B * pages * v.nkv < (1ll << 31) && ((long long)q.max_new * group <= kMaxCols || kv8_chunk_fits(v, q, group, pages));
}

cudaError_t kv8_attention(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                          int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, void* work, cudaStream_t s) {
  // the fewest n-tiles that hold every session's columns
  const long long cols = (long long)q.max_new * group;
  float* part = (float*)((char*)work + kCtas * (size_t)sms * sizeof(unsigned));
  // 9 to 16 columns of tiles that would be cut: the join of that many columns costs more
  // than the tensor cores' kernel while the work is small (8 rows of 2 q heads a kv head
  // behind 1000 tokens 27 and 19 us, 16 sessions of them 34 and 23; 8 sessions behind
  // 2000 31 and 27, behind 8000 50 and 68). The host knows no lengths: pages is what the
  // tables could hold, so short sessions in tables for long ones take the slower side (the
  // first two from tables of 2500 pages 27 and 34 us).
  const long long tiles = (long long)q.B * v.nkv, pages = most_pages(v, q);
  const bool whole = tiles <= sms * kCtas && pages <= (2 * tiles >= sms * kCtas ? kWholePagesMany : kWholePages);
  if (cols > kMaxCols || (cols > 8 && !whole && tiles * pages <= 128ll * sms && kv8_chunk_fits(v, q, group, pages)))
    return kv8_chunk(v, q, d, group, sms, qp, q_stride, scale, out, out_stride, (unsigned*)work, part, s);
  const int nt = cols <= 8 ? 1 : 2;
  Args a{};
  a.c = v;
  a.q = q;
  a.group = group;
  a.max_cols = (int)cols;
  a.one_each = (long long)q.B * v.nkv <= sms * kCtas;
  a.qp = qp;
  a.q_stride = q_stride;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.out_stride = out_stride;
  a.arrived = (unsigned*)work;
  a.part = part;
  if (d == 64)
    return nt == 1 ? launch_one<64, 1>(a, sms, s) : launch_one<64, 2>(a, sms, s);
  return nt == 1 ? launch_one<128, 1>(a, sms, s) : launch_one<128, 2>(a, sms, s);
}

}  // namespace qtts
