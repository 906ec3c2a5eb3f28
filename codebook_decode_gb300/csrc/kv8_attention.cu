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
// The work (tiles x their pages, in units of one page of one kv head) is cut
// into equal shares, one per CTA, whatever the sessions' lengths; a tile that
// several CTAs share is joined by the last of them to arrive, in CTA order, so
// results do not depend on which CTA that is.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv8.cuh"

namespace qtts {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsA = kWarps * 32;
constexpr float kSlack = 6.f;
constexpr float kNone = -1.5e38f;  // running maximum before the first value
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWaitTries = 1 << 20;  // bound of each wait for a copy (a try suspends for microseconds)

__host__ __device__ constexpr int ctas_per_sm(int NT) { return NT <= 2 ? 2 : 1; }
constexpr int kMaxCols = 32;

template <int D, int NT>
struct Smem {
  static constexpr int kSlots = (NT <= 2 ? 2 : 3) * (128 / D);
  static constexpr int kStride = D + 4;  // comb row in floats: a lane quad's 16-byte stores fall on different banks
  alignas(128) uint8_t ring[kWarps][kSlots][32 * D];
  alignas(16) float comb[kWarps / 2][8 * NT][kStride];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  float mj[8 * NT], lj[8 * NT];  // the warps' joined maximum and sum
  uint64_t bar[kWarps][kSlots];
  int flag, max_tile;
  long long cum[1];  // [B + 1] units before session b
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ bool wait_copy(uint64_t* bar, uint32_t parity) {
  for (int tries = 0; tries < kWaitTries; ++tries)
    if (mbar_test(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four codes to two half pairs: a byte under the exponent of 2^10 is 1024 +
// byte, minus 1152 the code itself, exactly.
__device__ __forceinline__ void widen(uint32_t c, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(c, 0x64646464u, 0x4140), b = __byte_perm(c, 0x64646464u, 0x4342);
  const uint32_t off = 0x64806480u;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(off));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(off));
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
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *(const uint32_t*)&h;
}

struct Args {
  Kv8View c;
  Kv8Batch q;
  int group, rows_per_tile;
  const uint16_t* qp;
  int64_t q_stride;
  float scale_log2;
  uint16_t* out;
  int64_t out_stride;
  float* part;        // [2 G] partial tiles: [cols][D] values, then m and l
  unsigned* arrived;  // [G] CTAs of the tile that starts in this CTA and ends in a later one; zero between calls
};
__host__ __device__ constexpr int part_floats(int D) { return kMaxCols * (D + 2); }

// pages that the last row of tile t sees
__device__ __forceinline__ int tile_pages(const Kv8Session& s, int t, int rows_per_tile) {
  return (s.L + min((t + 1) * rows_per_tile, s.n) + kPage - 1) / kPage;
}

// Where a unit lies: session b, kv head h, tile t, page p of it.
struct Place {
  int b, h, t, p, pages;
  Kv8Session s;
};
__device__ __forceinline__ Place place_of(const Args& a, const long long* cum, long long u) {
  Place r;
  int lo = 0, hi = a.q.B;  // cum[lo] <= u < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= u) lo = mid;
    else hi = mid;
  }
  r.b = lo;
  r.s = kv8_session(a.q, lo, a.c.max_context, a.c.err);
  const long long per = (cum[lo + 1] - cum[lo]) / a.c.nkv;
  long long rem = u - cum[lo];
  r.h = (int)(rem / per);
  rem -= r.h * per;
  r.t = 0;
  r.pages = tile_pages(r.s, 0, a.rows_per_tile);
  while (rem >= r.pages) {
    rem -= r.pages;
    r.pages = tile_pages(r.s, ++r.t, a.rows_per_tile);
  }
  r.p = (int)rem;
  return r;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreadsA, ctas_per_sm(NT)) attention_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using S = Smem<D, NT>;
  S& sm = *(S*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int KC = D / 64;   // 64-dim chunks of a K row
  constexpr int VJ = D / 32;   // 16-byte V words of a lane
  constexpr uint32_t kBytes = 32 * D;

  // shares: units before each session, then this CTA's range
  if (lane == 0)
    for (int i = 0; i < S::kSlots; ++i) mbar_init(&sm.bar[warp][i], 1);
  if (warp == 0) {
    long long carry = 0;
    int most = 0;
    for (int b0 = 0; b0 < a.q.B; b0 += 32) {
      long long w = 0;
      if (b0 + lane < a.q.B) {
        const Kv8Session s = kv8_session(a.q, b0 + lane, a.c.max_context, a.c.err);
        for (int t = 0; t * a.rows_per_tile < s.n; ++t) {
          const int p = tile_pages(s, t, a.rows_per_tile);
          w += p;
          most = max(most, p);
        }
        w *= a.c.nkv;
      }
      long long x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < a.q.B) sm.cum[b0 + lane] = carry + x - w;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      sm.cum[a.q.B] = carry;
      sm.max_tile = most;
      mbar_init_fence();
    }
  }
  __syncthreads();
  const long long total = sm.cum[a.q.B];
  // a share below two pages a warp (or a whole short tile) costs more in joining than it saves
  const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)min(sm.max_tile, 2 * kWarps));
  const long long u0 = blockIdx.x * share;
  if (u0 >= total) return;
  const int units = (int)(min(u0 + share, total) - u0);

  // This warp's units are i = warp + 8 n, n = 0, 1, ...; lane x holds the block
  // and scales of n = 32 k + x, and those of the next 32 are fetched meanwhile.
  auto fetch_block = [&](int k) {
    const int i = warp + kWarps * (32 * k + lane);
    if (i >= units) return 0;
    const Place r = place_of(a, sm.cum, u0 + i);
    int page = a.q.bt[(size_t)r.b * a.q.bt_stride + r.p];
    if (page < 0 || page >= a.c.pool_pages) {
      set_err(a.c.err, QTTS_DEV_BAD_PAGE);
      page = 0;  // inside the pool; the session's result is not used
    }
    return page * a.c.nkv + r.h;
  };
  auto fetch_scale = [&](int blk) { return *(const float2*)(a.c.scales + 2 * (size_t)blk); };
  int blk = fetch_block(0), blk_next = 0;
  float2 scl = fetch_scale(blk), scl_next = make_float2(0.f, 0.f);
  int n = 0;  // units this warp has done: slot n % kSlots, parity n / kSlots
  bool dead = false;
  // copy the block of this warp's unit k (at most kSlots ahead of n)
  auto issue = [&](int k) {
    const int from = __shfl_sync(0xffffffffu, (k ^ n) & 32 ? blk_next : blk, k & 31);
    if (lane == 0 && !dead && warp + kWarps * k < units) {
      uint64_t* bar = &sm.bar[warp][k % S::kSlots];
      mbar_arrive_expect_tx(bar, kBytes);
      bulk_load(sm.ring[warp][k % S::kSlots], a.c.codes + (size_t)from * kBytes, kBytes, bar);
    }
  };
#pragma unroll
  for (int k = 0; k < S::kSlots; ++k) issue(k);

  {
    int seg = 0;
    while (seg < units) {
      const Place r = place_of(a, sm.cum, u0 + seg);
      const int seg_end = min(units, seg + r.pages - r.p);
      const int row0 = r.t * a.rows_per_tile;
      const int rows = min(a.rows_per_tile, r.s.n - row0);
      const int cols = rows * a.group;

      // queries: rotated, scaled by a power of two per column, as B fragments
      uint32_t qf[NT][KC * 4][2];
      float cf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = nt * 8 + g;
        const int qr = col / a.group;  // row of the tile
        float x[KC][16];
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[c][e] = 0.f;
        if (col < cols) {
          const uint16_t* src = a.qp + (int64_t)(r.s.r0 + row0 + qr) * a.q_stride +
                                (size_t)(r.h * a.group + col - qr * a.group) * D + 16 * t4;
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 w = *(const uint2*)(src + 64 * c + 4 * e);
              x[c][4 * e] = bf2f(w.x & 0xffffu);
              x[c][4 * e + 1] = __uint_as_float(w.x & 0xffff0000u);
              x[c][4 * e + 2] = bf2f(w.y & 0xffffu);
              x[c][4 * e + 3] = __uint_as_float(w.y & 0xffff0000u);
            }
        }
        if (a.c.rope_cos) {
          const int pos = r.s.L + min(row0 + qr, r.s.n - 1);
          const size_t at = (size_t)pos * (D / 2) + 16 * (D == 128 ? t4 : t4 & 1);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 cs4 = *(const float4*)(a.c.rope_cos + at + e), sn4 = *(const float4*)(a.c.rope_sin + at + e);
            const float* cs = &cs4.x;
            const float* sn = &sn4.x;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              if constexpr (D == 128) {
                const float u = x[0][e + f], w = x[1][e + f];
                x[0][e + f] = u * cs[f] - w * sn[f];
                x[1][e + f] = w * cs[f] + u * sn[f];
              } else {  // the partner dim stands two lanes further
                const float u = x[0][e + f], w = __shfl_xor_sync(0xffffffffu, u, 2);
                x[0][e + f] = t4 < 2 ? u * cs[f] - w * sn[f] : u * cs[f] + w * sn[f];
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
        for (int e = 0; e < 2; ++e) see[nt][e] = r.s.L + row0 + min((nt * 8 + 2 * t4 + e) / a.group, rows - 1);
      const int first_masked = (r.s.L + row0 + 1) / kPage;  // pages before this one are seen whole by every row

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

      for (int i; (i = warp + kWarps * n) < seg_end; ++n) {
        if ((n & 31) == 0) {
          if (n) {
            blk = blk_next;
            scl = scl_next;
          }
          blk_next = fetch_block((n >> 5) + 1);
        } else if ((n & 31) == 16) {
          scl_next = fetch_scale(blk_next);
        }
        const int slot = n % S::kSlots;
        const uint32_t parity = (n / S::kSlots) & 1;
        if (!dead && !__all_sync(0xffffffffu, wait_copy(&sm.bar[warp][slot], parity))) {
          // no more copies; those in flight get one more wait, so that none lands after the CTA has left
          dead = true;
          set_err(a.c.err, QTTS_DEV_TIMEOUT);
          for (int k = n; k < n + S::kSlots; ++k)
            if (warp + kWarps * k < units) wait_copy(&sm.bar[warp][k % S::kSlots], (k / S::kSlots) & 1);
        }
        const uint8_t* kb = sm.ring[warp][slot];
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
        issue(n + S::kSlots);

        const float2 sc = make_float2(__shfl_sync(0xffffffffu, scl.x, n & 31), __shfl_sync(0xffffffffu, scl.y, n & 31));
        const float lv = lg2(fmaxf(sc.y, kKv8MinScale)) + (sc.y != sc.y ? sc.y : 0.f);
        const int page = r.p + i - seg;
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
          pf[nt][0] = transpose8(half2_bits(p[0] * sc.y, p[1] * sc.y));
          pf[nt][1] = transpose8(half2_bits(p[2] * sc.y, p[3] * sc.y));
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

      // join the warps: common maximum, weighted sums
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[nt][e];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
          if (g == 0) {
            sm.m[warp][nt * 8 + 2 * t4 + e] = m[nt][e];
            sm.l[warp][nt * 8 + 2 * t4 + e] = x;
          }
        }
      __syncthreads();
      if (tid < cols) {
        float mx = sm.m[0][tid], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][tid]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += ex2(sm.m[w][tid] - mx) * sm.l[w][tid];
        sm.mj[tid] = mx;
        sm.lj[tid] = sum;
      }
      auto comb_rows = [&](bool add, int w) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = nt * 8 + 2 * t4 + e;
            if (col < cols) {
              float mx = sm.m[0][col];
#pragma unroll
              for (int k = 1; k < kWarps; ++k) mx = fmaxf(mx, sm.m[k][col]);
              const float f = ex2(m[nt][e] - mx);
#pragma unroll
              for (int j = 0; j < VJ; ++j) {
                float4* dst = (float4*)&sm.comb[w][col][32 * j + 4 * g];
                float4 x = make_float4(o[nt][2 * j][e] * f, o[nt][2 * j][e + 2] * f, o[nt][2 * j + 1][e] * f,
                                       o[nt][2 * j + 1][e + 2] * f);
                if (add) {
                  const float4 y = *dst;
                  x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                }
                *dst = x;
              }
            }
          }
      };
      if (warp >= kWarps / 2) comb_rows(false, warp - kWarps / 2);
      __syncthreads();
      if (warp < kWarps / 2) comb_rows(true, warp);
      __syncthreads();

      // a whole tile is written; of a shared one each CTA leaves a partial, and
      // the last to arrive joins them in CTA order
      const long long ub = u0 + seg - r.p;  // the tile's units: [ub, ub + pages)
      const int c0 = (int)(ub / share), pieces = (int)((ub + r.pages - 1) / share) - c0 + 1;
      auto write = [&](int col, int x, float4 v, float sum) {
        const int qr = col / a.group;
        uint16_t* dst = a.out + (int64_t)(r.s.r0 + row0 + qr) * a.out_stride +
                        (size_t)(r.h * a.group + col - qr * a.group) * D + x;
        *(uint2*)dst = make_uint2(f2bf(v.x / sum) | (uint32_t)f2bf(v.y / sum) << 16,
                                  f2bf(v.z / sum) | (uint32_t)f2bf(v.w / sum) << 16);
      };
      // a CTA starts at most one shared tile and ends at most one that began earlier
      auto part_of = [&](int c) { return a.part + (size_t)(2 * c + (c == c0)) * part_floats(D); };
      float* part = part_of(blockIdx.x);
      for (int idx = tid; idx < cols * (D / 4); idx += kThreadsA) {
        const int col = idx / (D / 4), x = idx % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps / 2; ++w) {
          const float4 y = *(const float4*)&sm.comb[w][col][x];
          v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
        }
        if (pieces == 1) {
          write(col, x, v, sm.lj[col]);
        } else {
          *(float4*)(part + col * D + x) = v;
          if (x == 0) *(float2*)(part + kMaxCols * D + 2 * col) = make_float2(sm.mj[col], sm.lj[col]);
        }
      }
      if (pieces > 1) {
        __threadfence();
        __syncthreads();
        if (tid == 0) sm.flag = atomicAdd(&a.arrived[c0], 1u) == (unsigned)pieces - 1;
        __syncthreads();
        if (sm.flag) {
          __threadfence();
          for (int idx = tid; idx < cols * (D / 4); idx += kThreadsA) {
            const int col = idx / (D / 4), x = idx % (D / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            float mx = kNone, sum = 0.f;
#pragma unroll 4
            for (int p = 0; p < pieces; ++p) {
              const float* src = part_of(c0 + p);
              const float4 y = __ldcg((const float4*)(src + col * D + x));
              const float2 ml = __ldcg((const float2*)(src + kMaxCols * D + 2 * col));
              const float nm = fmaxf(mx, ml.x), f0 = ex2(mx - nm), f1 = ex2(ml.x - nm);
              mx = nm;
              sum = sum * f0 + ml.y * f1;
              v = make_float4(v.x * f0 + y.x * f1, v.y * f0 + y.y * f1, v.z * f0 + y.z * f1, v.w * f0 + y.w * f1);
            }
            write(col, x, v, sum);
          }
          if (tid == 0) a.arrived[c0] = 0;  // ready for the next call
        }
      }
      __syncthreads();  // the joined values have been read
      seg = seg_end;
    }
  }
}

template <int D, int NT>
size_t smem_bytes(int B) {
  return sizeof(Smem<D, NT>) + B * sizeof(long long);
}
template <int D, int NT>
cudaError_t setup_one() {
  return cudaFuncSetAttribute(attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_bytes<D, NT>(kKv8MaxBatch));
}
template <int D, int NT>
cudaError_t launch_one(const Args& a, int sms, cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(sms * ctas_per_sm(NT));
  lc.blockDim = dim3(kThreadsA);
  lc.dynamicSmemBytes = smem_bytes<D, NT>(a.q.B);
  lc.stream = s;
  return cudaLaunchKernelEx(&lc, attention_kernel<D, NT>, a);
}

}  // namespace

cudaError_t kv8_attention_setup(int d) {
  cudaError_t e;
  if (d == 64) {
    (e = setup_one<64, 1>()) || (e = setup_one<64, 2>()) || (e = setup_one<64, 4>());
  } else {
    (e = setup_one<128, 1>()) || (e = setup_one<128, 2>()) || (e = setup_one<128, 4>());
  }
  return e;
}

size_t kv8_attention_workspace(int d, int sms) {
  const size_t ctas = 2 * (size_t)sms;
  return ctas * sizeof(unsigned) + 2 * ctas * part_floats(d) * sizeof(float);
}

cudaError_t kv8_attention(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                          int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, void* work, cudaStream_t s) {
  // the fewest n-tiles that hold every session's columns; more rows go in tiles of 32 columns
  const long long cols = (long long)q.max_new * group;
  const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
  Args a{v,  q, group, 8 * nt / group, qp, q_stride, scale * kLog2e, out, out_stride, nullptr, (unsigned*)work};
  a.part = (float*)((char*)work + 2 * (size_t)sms * sizeof(unsigned));
  if (d == 64)
    return nt == 1 ? launch_one<64, 1>(a, sms, s) : nt == 2 ? launch_one<64, 2>(a, sms, s) : launch_one<64, 4>(a, sms, s);
  return nt == 1 ? launch_one<128, 1>(a, sms, s) : nt == 2 ? launch_one<128, 2>(a, sms, s) : launch_one<128, 4>(a, sms, s);
}

}  // namespace qtts
