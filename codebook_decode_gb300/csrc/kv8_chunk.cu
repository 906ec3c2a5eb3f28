// kv8_chunk.cu -- attention of many query rows over the 8-bit paged K/V cache,
// on the tcgen05 tensor cores (prompts, and batches with prompts among them).
//
// A tile is up to 128 rows (query tokens x the q heads of one kv head) of one
// session. For every 128 keys (8 pages)
//   S [128 x 128] = Q . K^T,   O [128 x d] += P . V
// with the accumulators in tensor memory and Q, K, V and P as half in shared
// memory, in the canonical K-major layout without swizzle. Codes are exact in
// half; the blocks' scales act outside the products, as in kv8_attention.cu:
// the K scale on the scores, the V scale on the weights.
//
// Warps: two softmax groups of four (a thread per row), which take the key
// steps in turn, each with its own S, P, O, maximum and sum, so that one
// group's softmax runs beside the other's products; four warps that widen the
// codes of the step after into shared memory (once per 128 rows); and one
// thread that issues the products. The two groups' results are joined at the
// tile's end. Bound by the softmax and widening instructions next to the
// products: 128 x 128 scores cost an SM about 1000 cycles of exponentials
// alone, the two products about 1300.
//
// Work is cut into equal shares of key steps, one per CTA; tiles that several
// CTAs share are joined through the workspace by the last to arrive, in order.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace qtts {
namespace {

constexpr int kRows = 128, kKeys = 128, kPagesPerStep = kKeys / kPage;
constexpr int kSoftmaxThreads = 256, kWidenThreads = 128;
constexpr int kThreadsC = kSoftmaxThreads + kWidenThreads + 32;
constexpr int kChunkTries = 1 << 20;

template <int D>
struct ChunkSmem {
  alignas(1024) uint8_t q[kRows * D * 2];
  uint8_t p[2][kRows * kKeys * 2];
  uint8_t k[2][kKeys * D * 2];
  uint8_t v[2][kKeys * D * 2];
  float2 ml[2][kRows];   // each group's maximum and sum; before the first step the rows' magnitudes
  float2 sc[4][kPagesPerStep];
  // kfull, vfull: widened; sdone: the step's scores are there (and its K place is free); pfull: its
  // weights; pvdone: its second product has run (V and P
  // places free); qfull: the tile's queries; drained: after a failure, all products issued
  uint64_t kfull[2], vfull[2], sdone[2], pfull[2], pvdone[2], qfull, drained;
  uint32_t tmem;
  int failed, verdict, flag, share, start_b, start_rem, total;
};

struct ChunkArgs {
  Kv8View c;
  Kv8Batch q;
  int group, rows_per_tile;
  const uint16_t* qp;
  int64_t q_stride;
  float scale_log2, q_sign;  // |softmax scale| log2 e, and its sign
  uint16_t* out;
  int64_t out_stride;
  float* part;        // [2 CTAs][kRows][D + 4]
  unsigned* arrived;  // [CTAs]
};

__device__ __forceinline__ int tile_steps(int L, int n, int t, int rows_per_tile) {
  return (L + min((t + 1) * rows_per_tile, n) + kKeys - 1) / kKeys;
}

// A place in the work: key step p of tile t of kv head h of session b.
struct Place {
  int b, h, t, p, steps;
  Kv8Session s;
  __device__ __forceinline__ void enter(const ChunkArgs& a, int bb) {
    for (b = bb; b < a.q.B; ++b) {
      s = kv8_session(a.q, b, a.c.max_context, a.c.err);
      if (s.n) break;
    }
    h = t = p = 0;
    steps = b < a.q.B ? tile_steps(s.L, s.n, 0, a.rows_per_tile) : 0x7fffffff;
  }
  __device__ __forceinline__ void next_tile(const ChunkArgs& a) {
    p = 0;
    if ((t + 1) * a.rows_per_tile < s.n) {
      ++t;
    } else {
      t = 0;
      if (++h == a.c.nkv) {
        enter(a, b + 1);
        return;
      }
    }
    steps = tile_steps(s.L, s.n, t, a.rows_per_tile);
  }
};

__device__ __forceinline__ int session_steps(const ChunkArgs& a, int b) {
  if (b >= a.q.B) return 0;
  const Kv8Session s = kv8_session(a.q, b, a.c.max_context, a.c.err);
  int w = 0;
  for (int t = 0; t * a.rows_per_tile < s.n; ++t) w += tile_steps(s.L, s.n, t, a.rows_per_tile);
  return w * a.c.nkv;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
constexpr uint32_t idesc_f16(int M, int N) {  // kind::f16: fp32 accumulator, half A and B, both K-major
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t (&r)[8], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The order in which a page's 16 tokens stand along the key axis of both
// products: that of the V blocks' words. Place n holds token_of(n).
__host__ __device__ constexpr int token_of(int n) { return 2 * (n >> 2) + (n & 1) + ((n >> 1) & 1) * 8; }

template <int D>
__global__ void __launch_bounds__(kThreadsC, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem<D>& sm = *(ChunkSmem<D>*)smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kCol = D + 4;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kfull[i], kWidenThreads);
      mbar_init(&sm.vfull[i], kWidenThreads);
      mbar_init(&sm.sdone[i], 1);
      mbar_init(&sm.pfull[i], kSoftmaxThreads / 2);
      mbar_init(&sm.pvdone[i], 1);
    }
    mbar_init(&sm.qfull, kSoftmaxThreads);
    mbar_init(&sm.drained, 1);
    mbar_init_fence();
    sm.failed = 0;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {  // shares, and the session in which this CTA's begins
    int total = 0;
    for (int b0 = 0; b0 < a.q.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, session_steps(a, b0 + lane));
    const int share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, 4);
    const long long u0 = (long long)blockIdx.x * share;
    int carry = 0;
    for (int b0 = 0; b0 < a.q.B && u0 < total; b0 += 32) {
      int x = session_steps(a, b0 + lane);
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const long long lo = (long long)carry + x - own;
      if (lo <= u0 && u0 < lo + own) {
        sm.start_b = b0 + lane;
        sm.start_rem = (int)(u0 - lo);
      }
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      sm.share = share;
      sm.total = total;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int share = sm.share;
  const long long u0 = (long long)blockIdx.x * share;
  const int units = u0 < sm.total ? (int)min((long long)share, sm.total - u0) : 0;
  Place w;
  if (units) {
    w.enter(a, sm.start_b);
    int rem = sm.start_rem, per = session_steps(a, w.b) / a.c.nkv;
    w.h = rem / per;
    rem -= w.h * per;
    while (rem >= w.steps) {
      rem -= w.steps;
      w.steps = tile_steps(w.s.L, w.s.n, ++w.t, a.rows_per_tile);
    }
    w.p = rem;
  }
  // bounded; once one wait has run out all others give up too
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (int tries = 0; tries < kChunkTries; ++tries) {
      if (mbar_test(bar, parity)) return true;
      if ((tries & 63) == 63 && *(volatile int*)&sm.failed) return false;
    }
    sm.failed = 1;
    set_err(a.c.err, QTTS_DEV_TIMEOUT);
    return false;
  };
  // accumulators: S of group x at 128 x, O at 256 + 128 x
  constexpr uint32_t kSbo = 128, kLboRow = kRows * 16, kLboV = D * 16;

  if (warp >= 8 && warp < 12) {
    // ---- widen: step j (counted over the CTA) into place j & 1
    const int t = tid - kSoftmaxThreads;
    int j = 0;
    bool ok = true;
    // K: a warp takes 2 pages of a step, a lane of a load 8 rows x 4 words
    const int wp = t >> 5;
    const int r8 = lane & 7, dch = lane >> 3;
    uint4 kr[D / 16], vr[D / 16];
    auto blocks = [&](const Place& x, int step, int* out) {  // this warp's pages of the step; -1: beyond the tile
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pg = step * kPagesPerStep + wp * 2 + i;
        const int last = (x.s.L + min((x.t + 1) * a.rows_per_tile, x.s.n) - 1) / kPage;
        out[i] = -1;
        if (pg <= last) {
          int page = a.q.bt[(size_t)x.b * a.q.bt_stride + pg];
          if (page < 0 || page >= a.c.pool_pages) {
            set_err(a.c.err, QTTS_DEV_BAD_PAGE);
            page = 0;
          }
          out[i] = page * a.c.nkv + x.h;
        }
      }
    };
    const uint4 none = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);  // codes of 0
    auto load_k = [&](const int* blk) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint8_t* src = a.c.codes + (size_t)max(blk[i], 0) * (32 * D) + c * 1024 + token_of(n8 * 8 + r8) * 64 + dch * 16;
            kr[(i * 2 + n8) * (D / 64) + c] = blk[i] >= 0 ? *(const uint4*)src : none;
          }
    };
    // V: lane x takes the 4 dims 4x.. (d = 64: half a warp per page) of 8 tokens (two words) at a time
    constexpr int D4 = D / 4;
    auto load_v = [&](const int* blk) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {  // d = 128: words t = 0..3; d = 64: t = 2 (lane / 16) + 0, 1
          const int x = lane % D4, tq = D == 128 ? e : 2 * (lane / D4) + e;
          const uint8_t* src = a.c.codes + (size_t)max(blk[i], 0) * (32 * D) + 16 * D + x * 64 + tq * 16;
          vr[i * (D / 32) + e] = blk[i] >= 0 ? *(const uint4*)src : none;
        }
    };
    static_assert(2 * 2 * (D / 64) <= D / 16 && 2 * (D / 32) <= D / 16, "registers of a step's words");
    auto load_scale = [&](const int* b) {
      float2 v = make_float2(0.f, 0.f);
      const int mine = lane == 0 ? b[0] : b[1];
      if (lane < 2 && mine >= 0) v = *(const float2*)(a.c.scales + 2 * (size_t)mine);
      return v;
    };
    Place x = w;  // the step whose block ids were asked for last
    int left = units, next[2] = {-1, -1};
    auto advance = [&]() {
      if (++x.p == x.steps) x.next_tile(a);
      blocks(x, x.p, next);
    };
    float2 sc, sc_next = make_float2(0.f, 0.f);
    if (left) {
      blocks(x, x.p, next);
      sc = load_scale(next);
      load_k(next);
      load_v(next);
      if (left > 1) advance();
    }
    for (; left; ++j, --left) {
      const int s = j & 1;
      const uint32_t free_parity = ((j >> 1) - 1) & 1;
      if (j >= 2) ok = wait(&sm.sdone[s], free_parity);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane < 2) sm.sc[j & 3][wp * 2 + lane] = sc;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 k = kr[(i * 2 + n8) * (D / 64) + c];
            uint4 lo, hi;  // dims 64 c + 16 dch + 0..7, 8..15
            widen(k.x, lo.x, lo.y);
            widen(k.y, lo.z, lo.w);
            widen(k.z, hi.x, hi.y);
            widen(k.w, hi.z, hi.w);
            const int row8 = (wp * 2 + i) * 2 + n8, d8 = 8 * c + 2 * dch;
            uint8_t* dst = sm.k[s] + (d8 * (kKeys / 8) + row8) * 128 + r8 * 16;
            *(uint4*)dst = lo;
            *(uint4*)(dst + kLboRow) = hi;
          }
      fence_async_shared();
      mbar_arrive(&sm.kfull[s]);
      if (left > 1) {
        load_k(next);
        sc_next = load_scale(next);
      }
      if (j >= 2) ok = wait(&sm.pvdone[s], free_parity);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // row r = (D / 4) jd + x4 of the V operand holds dim 4 x4 + jd
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const int x4 = lane % D4, key8 = (wp * 2 + i) * 2 + (D == 128 ? h : lane / D4);
          const uint4 v0 = vr[i * (D / 32) + 2 * h], v1 = vr[i * (D / 32) + 2 * h + 1];
          const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int jd = 0; jd < 4; ++jd) {
            uint4 o;
            widen(w0[jd], o.x, o.y);
            widen(w1[jd], o.z, o.w);
            const int r = jd * D4 + x4;
            *(uint4*)(sm.v[s] + (key8 * (D / 8) + r / 8) * 128 + r % 8 * 16) = o;
          }
        }
      fence_async_shared();
      mbar_arrive(&sm.vfull[s]);
      if (left > 1) load_v(next);
      if (left > 2) advance();
      sc = sc_next;
    }
  } else if (warp == 12) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t idS = idesc_f16(kRows, kKeys), idO = idesc_f16(kRows, D);
      const uint32_t qa = smem_addr(sm.q);
      int j = 0, seg = 0, left = units;
      bool ok = true;
      auto scores = [&](int jj) {
        const int s = jj & 1;
        if (!(ok = wait(&sm.kfull[s], (jj >> 1) & 1))) return;
        tc_fence_after();
        const uint32_t ka = smem_addr(sm.k[s]);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma(tmem + 128 * s, tc_smem_desc(qa + ks * 2 * kLboRow, kLboRow, kSbo),
                 tc_smem_desc(ka + ks * 2 * kLboRow, kLboRow, kSbo), idS, ks > 0);
        tc_commit(&sm.sdone[s]);
      };
      while (left && ok) {
        const int cnt = min(left, w.steps - w.p), j1 = j + cnt, j0 = j;
        ok = wait(&sm.qfull, seg & 1);
        tc_fence_after();
        if (ok) scores(j);
        if (ok && cnt > 1) scores(j + 1);
        for (; j < j1 && ok; ++j) {
          const int s = j & 1;
          ok = wait(&sm.pfull[s], (j >> 1) & 1) && wait(&sm.vfull[s], (j >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t pa = smem_addr(sm.p[s]), va = smem_addr(sm.v[s]);
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            tc_mma(tmem + 256 + 128 * s, tc_smem_desc(pa + ks * 2 * kLboRow, kLboRow, kSbo),
                   tc_smem_desc(va + ks * 2 * kLboV, kLboV, kSbo), idO, j - j0 >= 2 || ks > 0);
          tc_commit(&sm.pvdone[s]);
          if (j + 2 < j1) scores(j + 2);
        }
        left -= cnt;
        ++seg;
        w.p += cnt;
        if (w.p == w.steps) w.next_tile(a);
      }
      if (!ok) {  // what was issued has to end before the tensor memory is given back
        tc_commit(&sm.drained);
        for (int tries = 0; tries < kChunkTries; ++tries)
          if (mbar_test(&sm.drained, 0)) break;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: thread = row, group x takes the steps of its parity
    const int x = warp >> 2, row = tid & 127;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + 128 * x + quarter, to = tmem + 256 + quarter;
    int j = 0, left = units;
    bool ok = true;
    while (left && ok) {
      const int cnt = min(left, w.steps - w.p);
      const int row0 = w.t * a.rows_per_tile, rows = min(a.rows_per_tile, w.s.n - row0), cols = rows * a.group;
      const int qr = row / a.group;
      const bool valid = row < cols;
      const int pos = w.s.L + row0 + min(qr, rows - 1);  // last position that this row sees
      // this group's half of the row's query: dims D/4 x.. and their partners D/2 further
      float lo[D / 4], hi[D / 4];
      {
        const uint16_t* src = a.qp + (int64_t)(w.s.r0 + row0 + qr) * a.q_stride +
                              (size_t)(w.h * a.group + row - qr * a.group) * D + x * (D / 4);
#pragma unroll
        for (int e = 0; e < D / 4; e += 4) {
          uint2 l2 = make_uint2(0u, 0u), h2 = make_uint2(0u, 0u);
          if (valid) {
            l2 = *(const uint2*)(src + e);
            h2 = *(const uint2*)(src + D / 2 + e);
          }
          lo[e] = bf2f(l2.x & 0xffffu);
          lo[e + 1] = __uint_as_float(l2.x & 0xffff0000u);
          lo[e + 2] = bf2f(l2.y & 0xffffu);
          lo[e + 3] = __uint_as_float(l2.y & 0xffff0000u);
          hi[e] = bf2f(h2.x & 0xffffu);
          hi[e + 1] = __uint_as_float(h2.x & 0xffff0000u);
          hi[e + 2] = bf2f(h2.y & 0xffffu);
          hi[e + 3] = __uint_as_float(h2.y & 0xffff0000u);
        }
        if (a.c.rope_cos) {
          const size_t at = (size_t)pos * (D / 2) + x * (D / 4);
#pragma unroll
          for (int e = 0; e < D / 4; e += 4) {
            const float4 c4 = *(const float4*)(a.c.rope_cos + at + e), s4 = *(const float4*)(a.c.rope_sin + at + e);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const float u = lo[e + f], v = hi[e + f];
              lo[e + f] = u * cc[f] - v * ss[f];
              hi[e + f] = v * cc[f] + u * ss[f];
            }
          }
        }
      }
      uint32_t mxe = 0;
#pragma unroll
      for (int e = 0; e < D / 4; ++e)
        mxe = max(mxe, max(__float_as_uint(lo[e]) & 0x7f800000u, __float_as_uint(hi[e]) & 0x7f800000u));
      sm.ml[x][row].x = __uint_as_float(mxe);
      softmax_sync();
      mxe = max(mxe, __float_as_uint(sm.ml[x ^ 1][row].x));
      const uint32_t ex = min(max(mxe, 1u << 23), 253u << 23);
      const float inv = __uint_as_float((254u << 23) - ex) * a.q_sign;
      const float cf = __uint_as_float(ex) * a.scale_log2;
#pragma unroll
      for (int e = 0; e < D / 4; e += 8) {
        const int d8 = (x * (D / 4) + e) / 8;
        uint8_t* dst = sm.q + (d8 * (kRows / 8) + row / 8) * 128 + row % 8 * 16;
        *(uint4*)dst = make_uint4(half2_bits(lo[e] * inv, lo[e + 1] * inv), half2_bits(lo[e + 2] * inv, lo[e + 3] * inv),
                                  half2_bits(lo[e + 4] * inv, lo[e + 5] * inv), half2_bits(lo[e + 6] * inv, lo[e + 7] * inv));
        *(uint4*)(dst + D / 16 * kLboRow) =
            make_uint4(half2_bits(hi[e] * inv, hi[e + 1] * inv), half2_bits(hi[e + 2] * inv, hi[e + 3] * inv),
                       half2_bits(hi[e + 4] * inv, hi[e + 5] * inv), half2_bits(hi[e + 6] * inv, hi[e + 7] * inv));
      }
      fence_async_shared();
      tc_fence_before();  // the last tile's accumulators have been read
      mbar_arrive(&sm.qfull);

      float m = kNone, l = 0.f;
      int mine = 0;  // steps of this group in this tile
      const int first_masked = (w.s.L + row0 + 1) / kKeys;
      for (int i = 0; i < cnt && ok; ++i, ++j) {
        if ((j & 1) != x) continue;
        const uint32_t parity = (j >> 1) & 1;
        ok = wait(&sm.kfull[x], parity) && wait(&sm.sdone[x], parity);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int step = w.p + i;
        const bool masked = step >= first_masked;
        const int lim = pos - step * kKeys;  // keys of the step that the row sees: places <= lim
        const float2* sc = sm.sc[j & 3];
        // largest score (with the V scale's logarithm, see kv8_attention.cu)
        float mx = kNone;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(r, ts + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float g = -INFINITY;
            if (masked) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (32 * c + 16 * h + token_of(e) <= lim) g = fmaxf(g, __uint_as_float(r[16 * h + e]));
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) g = fmaxf(g, __uint_as_float(r[16 * h + e]));
            }
            const float2 s2 = sc[2 * c + h];
            const float lv = lg2(fmaxf(s2.y, kKv8MinScale));
            const float v = fmaf(g, s2.x * cf, lv);
            mx = fmaxf(mx, g > -INFINITY ? v : kNone);
          }
        }
        // the product before last of this group frees its weights' place and its O
        if (j >= 2) ok = wait(&sm.pvdone[x], ((j >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool grow = mx > m + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - mx) : 1.f;
          if (grow) m = mx;
          l *= f;
          if (mine) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(r, to + 128 * x + 32 * c);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st32(to + 128 * x + 32 * c, r);
            }
            tmem_wait_st();
          }
        }
        uint8_t* dst = sm.p[x] + row / 8 * 128 + row % 8 * 16;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(r, ts + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 s2 = sc[2 * c + h];
            const float f = s2.x * cf;
            float p[16], sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              p[e] = ex2(fmaf(__uint_as_float(r[16 * h + e]), f, -m));
              if (masked && 32 * c + 16 * h + token_of(e) > lim) p[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) sum += p[e];
            l += sum;
            // a page that the row does not see gives nothing, whatever its scale
            const float sv = masked && 32 * c + 16 * h > lim ? 0.f : s2.y;
#pragma unroll
            for (int q8 = 0; q8 < 2; ++q8)
              *(uint4*)(dst + (4 * c + 2 * h + q8) * kLboRow) =
                  make_uint4(half2_bits(p[8 * q8] * sv, p[8 * q8 + 1] * sv), half2_bits(p[8 * q8 + 2] * sv, p[8 * q8 + 3] * sv),
                             half2_bits(p[8 * q8 + 4] * sv, p[8 * q8 + 5] * sv), half2_bits(p[8 * q8 + 6] * sv, p[8 * q8 + 7] * sv));
          }
        }
        fence_async_shared();
        tc_fence_before();
        mbar_arrive(&sm.pfull[x]);
        ++mine;
      }
      // the group's last product
      if (ok && mine) {
        const int last = (j - 1 - (((j - 1) & 1) != x)) >> 1;
        ok = wait(&sm.pvdone[x], last & 1);
      }
      ok = __all_sync(0xffffffffu, ok);
      sm.ml[x][row] = make_float2(m, l);
      softmax_sync();
      if (tid == 0) sm.verdict = *(volatile int*)&sm.failed;  // one for all threads: they meet again below
      softmax_sync();
      if (sm.verdict) break;
      tc_fence_after();
      const float2 mlA = sm.ml[0][row], mlB = sm.ml[1][row];
      const float mj = fmaxf(mlA.x, mlB.x), fA = ex2(mlA.x - mj), fB = ex2(mlB.x - mj);
      const float sum = mlA.y * fA + mlB.y * fB;
      const bool hasA = cnt > 1 || ((j - 1) & 1) == 0, hasB = cnt > 1 || ((j - 1) & 1) == 1;
      const bool starts = w.p == 0, ends = w.p + cnt == w.steps;
      const long long ub = u0 + (units - left) - w.p;
      const int c0 = (int)(ub / share), pieces = (int)((ub + w.steps - 1) / share) - c0 + 1;
      float* part = a.part + ((size_t)(2 * blockIdx.x + starts) * kRows + row) * kCol;
      uint16_t* out = a.out + (int64_t)(w.s.r0 + row0 + qr) * a.out_stride + (size_t)(w.h * a.group + row - qr * a.group) * D;
      // this group writes half of the dims: columns jd D/4 + y of O hold dim 4 y + jd
#pragma unroll 1
      for (int y0 = x * (D / 8); y0 < (x + 1) * (D / 8); y0 += 8) {
        float o[4][8];
#pragma unroll
        for (int jd = 0; jd < 4; ++jd) {
          uint32_t rA[8], rB[8];
          if (hasA) tmem_ld8(rA, to + jd * (D / 4) + y0);
          if (hasB) tmem_ld8(rB, to + 128 + jd * (D / 4) + y0);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[jd][e] = 0.f;
            if (hasA) o[jd][e] = __uint_as_float(rA[e]) * fA;
            if (hasB) o[jd][e] = fmaf(__uint_as_float(rB[e]), fB, o[jd][e]);
          }
        }
        if (valid && starts && ends) {
          const float r = 1.f / sum;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *(uint2*)(out + 4 * (y0 + e)) = make_uint2(f2bf(o[0][e] * r) | (uint32_t)f2bf(o[1][e] * r) << 16,
                                                       f2bf(o[2][e] * r) | (uint32_t)f2bf(o[3][e] * r) << 16);
        } else if (valid) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *(float4*)(part + 4 * (y0 + e)) = make_float4(o[0][e], o[1][e], o[2][e], o[3][e]);
        }
      }
      if (!(starts && ends)) {
        if (valid && x == 0) *(float2*)(part + D) = make_float2(mj, sum);
        __threadfence();
        softmax_sync();
        if (tid == 0) {
          sm.flag = atomicAdd(&a.arrived[c0], 1u) == (unsigned)pieces - 1;
          if (sm.flag) a.arrived[c0] = 0;  // ready for the next call
        }
        softmax_sync();
        if (sm.flag) {
          __threadfence();
          for (int r = warp; r < cols; r += kSoftmaxThreads / 32) {
            auto partial = [&](int i) { return a.part + ((size_t)(2 * (c0 + i) + (i == 0)) * kRows + r) * kCol; };
            float mm = kNone, ss = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < pieces; i0 += 32) {
              const int i = i0 + lane;
              const float2 ml = i < pieces ? __ldcg((const float2*)(partial(i) + D)) : make_float2(kNone, 0.f);
              const float nm = fmaxf(mm, warp_max(ml.x)), f0 = ex2(mm - nm), f1 = ex2(ml.x - nm);
              mm = nm;
              ss = ss * f0 + warp_sum(ml.y * f1);
              v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
              for (int k = 0; k < 32 && i0 + k < pieces; k += 4) {
                float4 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (lane < D / 4 && i0 + k + e < pieces) y[e] = __ldcg((const float4*)(partial(i0 + k + e) + 4 * lane));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) axpy(v, y[e], __shfl_sync(0xffffffffu, f1, k + e));
              }
            }
            if (lane < D / 4) {
              const int rq = r / a.group;
              const float inv_sum = 1.f / ss;
              uint16_t* o = a.out + (int64_t)(w.s.r0 + row0 + rq) * a.out_stride + (size_t)(w.h * a.group + r - rq * a.group) * D + 4 * lane;
              *(uint2*)o = make_uint2(f2bf(v.x * inv_sum) | (uint32_t)f2bf(v.y * inv_sum) << 16,
                                      f2bf(v.z * inv_sum) | (uint32_t)f2bf(v.w * inv_sum) << 16);
            }
          }
        }
      }
      left -= cnt;
      w.p += cnt;
      if (w.p == w.steps) w.next_tile(a);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

static_assert(sizeof(ChunkSmem<128>) <= 227 * 1024, "shared memory of a CTA");

template <int D>
cudaError_t launch_chunk(const ChunkArgs& a, int sms, cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(sms);
  lc.blockDim = dim3(kThreadsC);
  lc.dynamicSmemBytes = sizeof(ChunkSmem<D>);
  lc.stream = s;
  return cudaLaunchKernelEx(&lc, chunk_kernel<D>, a);
}

}  // namespace

cudaError_t kv8_chunk_setup(int d) {
  return d == 64 ? cudaFuncSetAttribute(chunk_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(ChunkSmem<64>))
                 : cudaFuncSetAttribute(chunk_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(ChunkSmem<128>));
}

size_t kv8_chunk_workspace(int d, int sms) { return 2 * (size_t)sms * kRows * (d + 4) * sizeof(float); }

cudaError_t kv8_chunk(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                      int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, unsigned* arrived, float* part,
                      cudaStream_t s) {
  ChunkArgs a{v, q, group, kRows / group, qp, q_stride, std::fabs(scale) * kLog2e, scale < 0.f ? -1.f : 1.f, out,
              out_stride, part, arrived};
  return d == 64 ? launch_chunk<64>(a, sms, s) : launch_chunk<128>(a, sms, s);
}

}  // namespace qtts
