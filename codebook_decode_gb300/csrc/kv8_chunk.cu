// kv8_chunk.cu -- attention of many query rows over the 8-bit paged K/V cache,
// on the tcgen05 tensor cores (prompts, and batches with prompts among them).
//
// A tile is up to 128 or 256 rows (query tokens x the q heads of one kv head)
// of one session. For every 128 keys (8 pages)
//   S [128 x 128] = Q . K^T,   O [128 x d] += P . V
// with the accumulators in tensor memory and Q, K, V and P as half in shared
// memory, K-major with the 128-byte swizzle. Codes are exact in
// half; the blocks' scales act outside the products, as in kv8_attention.cu:
// the K scale on the scores, the V scale on the weights.
//
// Warps: two softmax groups of four (a thread per row), four warps that widen
// the codes of the step after into shared memory, and one thread that issues
// the products. With 256 rows the groups have 128 each and a step's widened
// codes serve both; with 128 they take the steps in turn, each with its own S,
// P, O, maximum and sum, which are joined at the tile's end. Either way one
// group's softmax runs beside the other's products. Bound by the instructions
// of softmax and widening, which run next to the products.
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
constexpr int kSoftmaxThreads = 256, kWidenThreads = 256;
constexpr int kThreadsC = kSoftmaxThreads + kWidenThreads + 128;
// registers of a thread: launched, then of the softmax, widening and issuing groups
constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsWiden = 64, kRegsIssue = 64;
static_assert(kSoftmaxThreads * kRegsSoftmax + kWidenThreads * kRegsWiden + 128 * kRegsIssue <= kThreadsC * kRegsLaunch,
              "the groups share what the block was launched with");
constexpr int kChunkTries = 1 << 17;  // bound of each wait; a try sleeps up to about 10 us
constexpr int kJoinSteps = 6;
constexpr int kIssueWarp = (kSoftmaxThreads + kWidenThreads) / 32;

// Operands in shared memory: rows of 64 halves (128 bytes), rows one after the
// other, 64-wide blocks of columns one after the other, and in a row the 16-byte
// words exchanged by the row's low bits (the tensor cores' 128-byte swizzle), so
// that neither a row's words nor a word of neighbouring rows share banks (the
// unswizzled layout measured the same, with padding against bank conflicts).
__device__ __forceinline__ int word_at(int row, int word) { return row * 128 + ((word ^ (row & 7)) << 4); }
__device__ __forceinline__ uint64_t swizzled_desc(const void* p) {
  return (uint64_t)((smem_addr(p) >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// of the 16 columns (of k) number ks: their place in units of 16 bytes
__host__ __device__ constexpr uint64_t k_step(int ks, int rows) { return (ks / 4 * rows * 128 + ks % 4 * 32) / 16; }

template <int D, bool TWO>
struct ChunkSmem {
  alignas(1024) uint8_t q[TWO ? 2 : 1][kRows * D * 2];
  uint8_t p[2][kRows * kKeys * 2];
  uint8_t k[2][kKeys * D * 2];
  uint8_t v[TWO ? 1 : 2][kKeys * D * 2];
  float2 ml[2][kRows];  // each group's maximum and sum; before the first step the rows' query scales and offsets
  float4 sc[4][kPagesPerStep];  // a page's K scale, logarithm and reciprocal of its V scale
  // kfull, vfull: widened; kdone, vdone: read by the products; sdone: a group's
  // scores are there; pfull: its weights; pvdone: its second product has run;
  // qfull: the tile's queries; drained: after a failure, all products issued
  uint64_t kfull[2], vfull[2], kdone[2], vdone[2], sdone[2], pfull[2], pvdone[2], qfull, drained;
  uint32_t tmem;
  int failed, verdict, flag, share, whole, start_b, start_h, start_t, start_p, total;
};

struct ChunkArgs {
  Kv8View c;
  Kv8Batch q;
  int group, rows_per_tile, group_mul;  // r / group = r * group_mul >> 16 for r < 256
  const uint16_t* qp;
  int64_t q_stride;
  float scale_log2, q_sign;  // |softmax scale| log2 e, and its sign
  uint16_t* out;
  int64_t out_stride;
  float* part;        // [2 CTAs][tile rows][D + 4]
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
  __device__ __forceinline__ void advance(const ChunkArgs& a, int n) {
    p += n;
    while (p >= steps) {
      const int over = p - steps;
      next_tile(a);
      p = over;
    }
  }
};

// A session's tiles, weighed by their key steps (or 1 each: whole), up to the
// one that brings them past `limit`: returns that tile (or all tiles), `sum` the
// weight of those before it.
__device__ __forceinline__ int tiles_until(const Kv8Session& s, int rows_per_tile, bool whole, int limit, int& sum) {
  const int all = (s.n + rows_per_tile - 1) / rows_per_tile;
  if (whole) return sum = min(all, limit);
  int t = 0, keys = s.L + rows_per_tile + kKeys - 1;
  sum = 0;
#pragma unroll 1
  for (; t < all; ++t, keys += rows_per_tile) {
    const int here = t + 1 < all ? keys / kKeys : (s.L + s.n + kKeys - 1) / kKeys;
    if (sum + here > limit) break;
    sum += here;
  }
  return t;
}

template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
__device__ __forceinline__ void group_sync(int x) {  // one softmax group
  asm volatile("bar.sync %0, %1;" ::"r"(2 + x), "n"(kSoftmaxThreads / 2) : "memory");
}
template <int R>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t (&r)[8], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// codes 0, 1 and 2, 3 of four as 1024 + byte
__device__ __forceinline__ uint32_t raise_lo(uint32_t c) { return __byte_perm(c, 0x64646464u, 0x4140); }
__device__ __forceinline__ uint32_t raise_hi(uint32_t c) { return __byte_perm(c, 0x64646464u, 0x4342); }

// The order in which a page's 16 tokens stand along the key axis of both
// products: that of the V blocks' words. Place n holds token_of(n).
__host__ __device__ constexpr int token_of(int n) { return 2 * (n >> 2) + (n & 1) + ((n >> 1) & 1) * 8; }

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreadsC, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Smem = ChunkSmem<D, TWO>;
  Smem& sm = *(Smem*)smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kCol = D + 4;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kfull[i], kWidenThreads / 2);
      mbar_init(&sm.vfull[i], kWidenThreads / 2);
      mbar_init(&sm.kdone[i], 1);
      mbar_init(&sm.vdone[i], 1);
      mbar_init(&sm.sdone[i], 2);  // the products, and the issuing thread after it saw the codes' factors
      mbar_init(&sm.pfull[i], kSoftmaxThreads / 2);
      mbar_init(&sm.pvdone[i], 1);
    }
    mbar_init(&sm.qfull, kSoftmaxThreads);
    mbar_init(&sm.drained, 1);
    mbar_init_fence();
    sm.failed = 0;
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dependency_wait();
  if (warp == 0) {
    // Shares, and the place where this CTA's begins. Whole tiles where the most
    // that a CTA gets is not worse than an equal share and the cost of joining
    // cut tiles (reading queries twice, partials out and in: kJoinSteps).
    int total = 0, tiles = 0, most = 0, per = 0, own = 0, lo = 0, share = 0, rows = 0;
    bool whole = false;
    long long u0 = 0, u1 = 0;
    Kv8Session ses;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      int carry = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.q.B; b0 += 32) {
        if (!pass || a.q.B > 32) {
          ses.n = 0;
          if (b0 + lane < a.q.B) ses = kv8_session(a.q, b0 + lane, a.c.max_context, a.c.err);
        }
        const int count = tiles_until(ses, a.rows_per_tile, whole, 0x7fffffff, per);
        own = per * a.c.nkv;
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        lo = carry + x - own;
        carry += __shfl_sync(0xffffffffu, x, 31);
        if (!pass) {
          tiles += __reduce_add_sync(0xffffffffu, count * a.c.nkv);
          rows += __reduce_add_sync(0xffffffffu, ses.n);
          most = max(most, __reduce_max_sync(0xffffffffu, ses.n ? (ses.L + ses.n + kKeys - 1) / kKeys : 0));
        } else if (lo <= u0 && u0 < (long long)lo + own) {
          const int at = (int)(u0 - lo), h = at / per;
          int sum;
          sm.start_b = b0 + lane;
          sm.start_h = h;
          sm.start_t = tiles_until(ses, a.rows_per_tile, whole, at - h * per, sum);
          sm.start_p = at - h * per - sum;
        }
      }
      if (pass == 0) {
        // sessions that share rows (a row_start that goes back): the work would not be bounded by n_rows
        if (rows > a.q.n_rows) {
          set_err(a.c.err, QTTS_DEV_BAD_SESSION);
          break;
        }
        total = carry;
        const int G = gridDim.x;
        share = max((total + G - 1) / G, 4);
        whole = (long long)((tiles + G - 1) / G) * most <= share + kJoinSteps;
        u0 = whole ? (long long)tiles * blockIdx.x / G : (long long)blockIdx.x * share;
        u1 = whole ? (long long)tiles * (blockIdx.x + 1) / G : min(u0 + share, (long long)total);
        if (u0 >= u1) break;
      }
    }
    if (lane == 0) {
      sm.share = share;
      sm.whole = whole;
      sm.total = (int)max(u1 - u0, 0ll);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int share = sm.share;
  const long long u0 = (long long)blockIdx.x * share;  // of a cut
  int units = sm.total;  // key steps of this CTA
  Place w;
  if (units) {
    w.enter(a, sm.start_b);
    w.h = sm.start_h;
    w.t = sm.start_t;
    w.p = sm.start_p;
    w.steps = tile_steps(w.s.L, w.s.n, w.t, a.rows_per_tile);
    if (sm.whole) {
      Place x = w;
      const int tiles = units;
      units = 0;
      for (int i = 0; i < tiles; ++i) {
        units += x.steps;
        if (i + 1 < tiles) x.next_tile(a);
      }
    }
  }
  // bounded; once one wait has run out all others give up too
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
    for (int tries = 0; tries < kChunkTries; ++tries) {
      if (mbar_test_sleep(bar, parity, 10000)) return true;
      if (*(volatile int*)&sm.failed) return false;
    }
    sm.failed = 1;
    set_err(a.c.err, QTTS_DEV_TIMEOUT);
    return false;
  };
  auto row_of = [&](int r) { return r * a.group_mul >> 16; };  // a tile row's query row
  // accumulators: S of group x at 128 x, O at 256 + 128 x

  if (warp >= kSoftmaxThreads / 32 && warp < kIssueWarp) {
    set_regs_down<kRegsWiden>();
    // ---- widen: step j (counted over the CTA) into place j & 1
    // four warps for K, four for V, so that neither waits for the other's place;
    // a warp takes 2 of a step's pages
    const bool is_v = warp >= kSoftmaxThreads / 32 + 4;
    const int wp = (warp & 3) * 2;
    int j = 0;
    bool ok = true;
    // lane x holds the block of page x & 1 of this warp's two, of step 16 k + x / 2
    // (-1: beyond the tile); the next 16 steps' are fetched meanwhile
    Place ahead = w;
    auto fetch_ids = [&](int k) {
      int id = -1;
      if (16 * k + (lane >> 1) < units) {
        Place x = ahead;
        x.advance(a, lane >> 1);
        const int pg = x.p * kPagesPerStep + wp + (lane & 1);
        if (pg <= (x.s.L + min((x.t + 1) * a.rows_per_tile, x.s.n) - 1) / kPage) {
          int page = a.q.bt[(size_t)x.b * a.q.bt_stride + pg];
          if (page < 0 || page >= a.c.pool_pages) {
            set_err(a.c.err, QTTS_DEV_BAD_PAGE);
            page = 0;  // inside the pool; the session's result is not used
          }
          id = page * a.c.nkv + x.h;
        }
      }
      if (16 * (k + 1) < units) ahead.advance(a, 16);
      return id;
    };
    int left = units, ids = -1, ids_next = -1;
    // K: a lane of a load is one of 8 tokens x 4 words. V: lane x takes the 4 dims
    // 4x.. (d = 64: of half the words)
    constexpr int D4 = D / 4, kWords = D / 32;  // 16-byte words of a lane and page
    const int r8 = lane & 7, dch = lane >> 3, x4 = lane % D4;
    const size_t lane_at = is_v ? 16 * D + x4 * 64 + (D == 128 ? 0 : lane / D4 * 32) : dch * 16;
    uint4 wd[2][kWords];
    float2 sc[2];
    auto load = [&](int step) {
      const int from = (step ^ j) & 16 ? ids_next : ids;
      const uint4 none = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);  // codes of 0
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int id = __shfl_sync(0xffffffffu, from, 2 * (step & 15) + i);
        const uint8_t* src = a.c.codes + (size_t)max(id, 0) * (32 * D) + lane_at;
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const int at = is_v ? e * 16 : e % (D / 64) * 1024 + token_of(e / (D / 64) * 8 + r8) * 64;
          wd[i][e] = id >= 0 ? *(const uint4*)(src + at) : none;
        }
        sc[i] = !is_v && id >= 0 ? *(const float2*)(a.c.scales + 2 * (size_t)id) : make_float2(0.f, 0.f);
      }
    };
    if (left) {
      ids = fetch_ids(0);
      load(0);
    }
    for (; left; ++j, --left) {
      if ((j & 15) == 0 && j) ids = ids_next;
      if ((j & 15) == 8) ids_next = fetch_ids((j >> 4) + 1);
      const int s = j & 1;
      if (!is_v) {
        if (j >= 2) ok = wait(&sm.kdone[s], ((j >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane < 2) {
          const float2 v = lane ? sc[1] : sc[0];
          const float sv = v.y != v.y ? v.y : fmaxf(v.y, kKv8MinScale);
          sm.sc[j & 3][wp + lane] = make_float4(v.x, lg2(sv), 1.f / sv, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < kWords; ++e) {
            // as 1024 + byte: the score's surplus, 1152 times the query's sum, leaves in the softmax
            const uint4 k = wd[i][e];
            uint8_t* dst = sm.k[s] + e % (D / 64) * (kKeys * 128);
            const int row = (wp + i) * kPage + e / (D / 64) * 8 + r8;
            *(uint4*)(dst + word_at(row, 2 * dch)) = make_uint4(raise_lo(k.x), raise_hi(k.x), raise_lo(k.y), raise_hi(k.y));
            *(uint4*)(dst + word_at(row, 2 * dch + 1)) = make_uint4(raise_lo(k.z), raise_hi(k.z), raise_lo(k.w), raise_hi(k.w));
          }
      } else {
        const int vs = TWO ? 0 : s;
        if (j >= (TWO ? 1 : 2)) ok = wait(&sm.vdone[vs], TWO ? (j - 1) & 1 : ((j >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // row r = (D / 4) jd + x4 of the V operand holds dim 4 x4 + jd
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < kWords / 2; ++h) {
            const uint4 v0 = wd[i][2 * h], v1 = wd[i][2 * h + 1];
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int jd = 0; jd < 4; ++jd) {
              uint4 o;
              widen(w0[jd], o.x, o.y);
              widen(w1[jd], o.z, o.w);
              const int key8 = 2 * (wp + i) + (D == 128 ? h : lane / D4);
              *(uint4*)(sm.v[vs] + key8 / 8 * (D * 128) + word_at(jd * D4 + x4, key8 % 8)) = o;
            }
          }
      }
      fence_async_shared();
      mbar_arrive(is_v ? &sm.vfull[TWO ? 0 : s] : &sm.kfull[s]);
      if (left > 1) load(j + 1);
    }
  } else if (warp >= kIssueWarp) {
    // ---- products
    set_regs_down<kRegsIssue>();
    if (warp == kIssueWarp && lane == 0) {
      constexpr uint32_t idS = idesc_f16(kRows, kKeys), idO = idesc_f16(kRows, D);
      int j = 0, seg = 0, left = units, n[2] = {0, 0};  // n: steps of each group
      bool ok = true;
      auto scores = [&](int jj, int x, bool last) {  // group x's scores of step jj; last: K's place is free after
        const int s = jj & 1;
        if (!(ok = wait(&sm.kfull[s], (jj >> 1) & 1))) return;
        tc_fence_after();
        // a descriptor's low bits are the address in 16-byte units: steps along k add to it
        const uint64_t qd = swizzled_desc(sm.q[TWO ? x : 0]), kd = swizzled_desc(sm.k[s]);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma(tmem + 128 * x, qd + k_step(ks, kRows), kd + k_step(ks, kKeys), idS, ks > 0);
        tc_commit(&sm.sdone[x]);
        mbar_arrive(&sm.sdone[x]);
        if (last) tc_commit(&sm.kdone[s]);
      };
      auto weights_there = [&](int x) {  // group x has read its scores and written its weights
        ok = wait(&sm.pfull[x], n[x] & 1);
        ++n[x];
        return ok;
      };
      auto values = [&](int jj, int x, bool first, bool last) {  // group x's second product of step jj
        const int vs = TWO ? 0 : jj & 1;
        if (!(ok = wait(&sm.vfull[vs], TWO ? jj & 1 : (jj >> 1) & 1))) return;
        tc_fence_after();
        const uint64_t pd = swizzled_desc(sm.p[x]), vd = swizzled_desc(sm.v[vs]);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          tc_mma(tmem + 256 + 128 * x, pd + k_step(ks, kRows), vd + k_step(ks, D), idO, !first || ks > 0);
        tc_commit(&sm.pvdone[x]);
        if (last) tc_commit(&sm.vdone[vs]);
      };
      while (left && ok) {
        const int cnt = min(left, w.steps - w.p), j0 = j, j1 = j + cnt;
        ok = wait(&sm.qfull, seg & 1);
        tc_fence_after();
        if constexpr (TWO) {
          const bool both = min(a.rows_per_tile, w.s.n - w.t * a.rows_per_tile) * a.group > kRows;
#pragma unroll 1
          for (int x = 0; x <= both && ok; ++x) scores(j, x, x == both);
          for (; j < j1 && ok; ++j)
#pragma unroll 1
            for (int x = 0; x <= both && ok; ++x) {
              // the group's next scores first: it waits for them, not for the values
              if (weights_there(x) && j + 1 < j1) scores(j + 1, x, x == both);
              if (ok) values(j, x, j == j0, x == both);
            }
        } else {
#pragma unroll 1
          for (int i = 0; i < min(cnt, 2) && ok; ++i) scores(j + i, (j + i) & 1, true);
          for (; j < j1 && ok; ++j) {
            if (weights_there(j & 1) && j + 2 < j1) scores(j + 2, j & 1, true);
            if (ok) values(j, j & 1, j - j0 < 2, true);
          }
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
    // ---- softmax: thread = row; group x has its own rows, or takes the steps of its parity
    set_regs_up<kRegsSoftmax>();
    const int x = warp >> 2, row = tid & 127;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + 128 * x + quarter, to = tmem + 256 + quarter;
    int j = 0, left = units, n = 0;  // n: steps of this group
    bool ok = true;
    while (left && ok) {
      const int cnt = min(left, w.steps - w.p);
      const int row0 = w.t * a.rows_per_tile, rows = min(a.rows_per_tile, w.s.n - row0), cols = rows * a.group;
      const int pos = w.s.L + row0 + min(row_of(TWO ? tid : row), rows - 1);  // last position that this row sees
      const bool active = !TWO || x == 0 || cols > kRows;
      // The tile's queries, rotated, into shared memory. They and their rotations
      // are copied to the weights' place first, up to 128 rows at a time, all
      // copies in flight at once (loaded into registers they took a memory
      // latency for every few rows). A thread then takes 4 dims of a row and
      // their partners D/2 further, D/8 lanes a row. Scaled by the power of two
      // of the row's largest magnitude (before the rotation, which can grow it by
      // sqrt 2: half has room).
      constexpr int kQuads = D / 8, kRowsOnce = kSoftmaxThreads / kQuads;
      uint8_t* raw = sm.p[0];                    // [128][D] bf16
      uint8_t* turn = sm.p[0] + kRows * D * 2;   // [tokens][D / 2 cosines, D / 2 sines]; tokens x D x 4 <= 128 x D x 2
      const int pass_tokens = a.group > 1 ? kRows * a.group_mul >> 16 : kRows / 2;
#pragma unroll 1
      for (int tok = 0; tok < rows; tok += pass_tokens) {
        const int tokens = min(pass_tokens, rows - tok), first = tok * a.group, count = tokens * a.group;
        for (int i = tid; i < count * (D / 4); i += kSoftmaxThreads) {
          const int r = first + i / (D / 4), at = i % (D / 4) * 4, rq = row_of(r);
          copy_async<8>(raw + i * 8, a.qp + (int64_t)(w.s.r0 + row0 + rq) * a.q_stride + (size_t)(w.h * a.group + r - rq * a.group) * D + at);
        }
        if (a.c.rope_cos)
          for (int i = tid; i < tokens * (D / 4); i += kSoftmaxThreads) {
            const int at = i % (D / 8) * 4;
            const float* src = i / (D / 8) & 1 ? a.c.rope_sin : a.c.rope_cos;
            copy_async<16>(turn + i * 16, src + (size_t)(w.s.L + row0 + tok + i / (D / 4)) * (D / 2) + at);
          }
        asm volatile("cp.async.wait_all;" ::: "memory");
        softmax_sync();
        const int quad = tid % kQuads * 4;
        constexpr int U = 4;  // rows at once: their reductions over lanes overlap
#pragma unroll 1
        for (int r1 = tid / kQuads; r1 < kRows && r1 - tid / kQuads < count; r1 += U * kRowsOnce) {
          uint2 lo2[U], hi2[U];
          uint32_t mag[U];
#pragma unroll
          for (int k = 0; k < U; ++k) {  // rows beyond the last are what stands there: nothing reads them
            const uint8_t* src = raw + ((r1 + k * kRowsOnce) % kRows * D + quad) * 2;
            lo2[k] = *(const uint2*)src;
            hi2[k] = *(const uint2*)(src + D);
            mag[k] = __vmaxu2(__vmaxu2(lo2[k].x & 0x7fff7fffu, lo2[k].y & 0x7fff7fffu),
                              __vmaxu2(hi2[k].x & 0x7fff7fffu, hi2[k].y & 0x7fff7fffu));
            mag[k] = max(mag[k] & 0xffffu, mag[k] >> 16);
          }
#pragma unroll
          for (int o = 1; o < kQuads; o <<= 1)
#pragma unroll
            for (int k = 0; k < U; ++k) mag[k] = max(mag[k], __shfl_xor_sync(0xffffffffu, mag[k], o));
          float sum[U];  // of the rows' halves
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int rl = r1 + k * kRowsOnce, r = first + rl;
            const uint32_t ex = min(max(mag[k] << 16 & 0x7f800000u, 1u << 23), 253u << 23);
            const float inv = __uint_as_float((254u << 23) - ex) * a.q_sign;
            uint64_t p0 = pack2(__uint_as_float(lo2[k].x << 16) * inv, __uint_as_float(lo2[k].x & 0xffff0000u) * inv);
            uint64_t p1 = pack2(__uint_as_float(lo2[k].y << 16) * inv, __uint_as_float(lo2[k].y & 0xffff0000u) * inv);
            uint64_t q0 = pack2(__uint_as_float(hi2[k].x << 16) * inv, __uint_as_float(hi2[k].x & 0xffff0000u) * inv);
            uint64_t q1 = pack2(__uint_as_float(hi2[k].y << 16) * inv, __uint_as_float(hi2[k].y & 0xffff0000u) * inv);
            if (a.c.rope_cos) {
              const uint8_t* tr = turn + min(row_of(r) - tok, tokens - 1) * (D * 4) + quad * 4;
              const ulonglong2 cs = *(const ulonglong2*)tr;
              const float4 s4 = *(const float4*)(tr + D * 2);
              const uint64_t s0 = pack2(s4.x, s4.y), s1 = pack2(s4.z, s4.w), m0 = pack2(-s4.x, -s4.y), m1 = pack2(-s4.z, -s4.w);
              const uint64_t u0 = p0, u1 = p1;
              p0 = fma2(u0, cs.x, mul2(q0, m0));
              p1 = fma2(u1, cs.y, mul2(q1, m1));
              q0 = fma2(q0, cs.x, mul2(u0, s0));
              q1 = fma2(q1, cs.y, mul2(u1, s1));
            }
            const uint64_t val[4] = {p0, p1, q0, q1};
            uint32_t hu[4];
            float part[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const float2 y = unpack2(val[f]);
              hu[f] = half2_bits(y.x, y.y);
              const float2 z = __half22float2(*(const __half2*)&hu[f]);
              part[f] = z.x + z.y;
            }
            sum[k] = (part[0] + part[1]) + (part[2] + part[3]);
            if (rl < count) {
              // dims quad.. and D / 2 + quad..
              uint8_t* dst = sm.q[TWO ? r >> 7 : 0] + (quad & 4) * 2;
              *(uint2*)(dst + word_at(r & 127, quad / 8)) = make_uint2(hu[0], hu[1]);
              *(uint2*)(dst + (D == 128 ? kRows * 128 + word_at(r & 127, quad / 8) : word_at(r & 127, 4 + quad / 8))) = make_uint2(hu[2], hu[3]);
              if (quad == 0) sm.ml[TWO ? r >> 7 : 1][r & 127].x = __uint_as_float(ex) * a.scale_log2;
            }
          }
#pragma unroll
          for (int o = 1; o < kQuads; o <<= 1)
#pragma unroll
            for (int k = 0; k < U; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int rl = r1 + k * kRowsOnce, r = first + rl;
            if (quad == 0 && rl < count) sm.ml[TWO ? r >> 7 : 1][r & 127].y = 1152.f * sum[k];
          }
        }
        softmax_sync();  // before the next rows or the first weights take the place
      }
      const float cf = sm.ml[TWO ? x : 1][row].x, surplus = sm.ml[TWO ? x : 1][row].y;
      fence_async_shared();
      tc_fence_before();  // the last tile's accumulators have been read
      mbar_arrive(&sm.qfull);

      float m = kNone, l = 0.f;
      int mine = 0;  // steps of this group in this tile
      const int first_masked = (w.s.L + row0 + 1) / kKeys;
      for (int i = 0; i < cnt && ok; ++i, ++j) {
        if (TWO ? !active : (j & 1) != x) continue;
        ok = wait(&sm.sdone[x], n & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int step = w.p + i;
        const int lim = pos - step * kKeys;  // keys of the step that the row sees: those at <= lim
        const float4* sc = sm.sc[j & 3];
        const bool masked = step >= first_masked;
        uint32_t r[2][32];  // half of the row's scores at a time
        auto load_scores = [&](int half) {
          tmem_ld32(r[0], ts + 64 * half);
          tmem_ld32(r[1], ts + 64 * half + 32);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int n = 0; n < 64; ++n)
              if (64 * half + n / kPage * kPage + token_of(n % kPage) > lim) r[n / 32][n % 32] = 0xff800000u;  // -inf
          }
        };
        // a page's factors: of one that the row does not see at all they are
        // harmless ones, whatever its scales
        auto factors = [&](int page) {
          float4 f = sc[page];
          if (masked && page * kPage > lim) f = make_float4(1.f, 0.f, 1.f, 0.f);
          f.x = max_nan(f.x * cf, kKv8MinScale);  // positive: -inf stays -inf
          f.y = fmaf(-surplus, f.x, f.y);
          return f;
        };
        float mx = kNone;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          load_scores(half);
#pragma unroll
          for (int page = 0; page < kPagesPerStep / 2; ++page) {
            auto at = [&](int e) { return __uint_as_float(r[page / 2][page % 2 * 16 + e]); };
            float g = max3(at(0), at(1), at(2));
#pragma unroll
            for (int e = 3; e < 15; e += 2) g = max3(g, at(e), at(e + 1));
            g = fmaxf(g, at(15));
            const float4 f = factors(half * (kPagesPerStep / 2) + page);
            mx = fmaxf(mx, fmaf(g, f.x, f.y));
          }
        }
        // the product before last of this group frees its weights' place and its O
        if (n) ok = wait(&sm.pvdone[x], (n - 1) & 1);
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
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(o, to + 128 * x + 16 * c);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(to + 128 * x + 16 * c, o);
            }
            tmem_wait_st();
          }
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          load_scores(half);
#pragma unroll
          for (int page = 0; page < kPagesPerStep / 2; ++page) {
            const float4 f = factors(half * (kPagesPerStep / 2) + page);
            const uint64_t mul = pack2(f.x, f.x), off = pack2(f.y - m, f.y - m);
            uint64_t sum = 0;
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t* s2 = &r[page / 2][page % 2 * 16 + 2 * e];
              const float2 y = unpack2(fma2(pack2(__uint_as_float(s2[0]), __uint_as_float(s2[1])), mul, off));
              const float p0 = ex2(y.x), p1 = ex2(y.y);  // weight times V scale
              sum = add2(sum, pack2(p0, p1));
              h[e] = half2_bits(p0, p1);
            }
            const float2 t = unpack2(sum);
            l = fmaf(t.x + t.y, f.z, l);
            uint8_t* dst = sm.p[x] + half * (kRows * 128);
            *(uint4*)(dst + word_at(row, 2 * page)) = make_uint4(h[0], h[1], h[2], h[3]);
            *(uint4*)(dst + word_at(row, 2 * page + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        fence_async_shared();
        tc_fence_before();
        mbar_arrive(&sm.pfull[x]);
        ++mine;
        ++n;
      }
      if (ok && mine) ok = wait(&sm.pvdone[x], (n - 1) & 1);  // the group's last product
      ok = __all_sync(0xffffffffu, ok);
      sm.ml[x][row] = make_float2(m, l);
      softmax_sync();
      if (tid == 0) sm.verdict = *(volatile int*)&sm.failed;  // one for all threads: they meet again below
      softmax_sync();
      if (sm.verdict) break;
      tc_fence_after();
      // the row's maximum and sum; with both groups on the same rows their factors, and the joined ones
      float fA = 1.f, fB = 1.f;
      float2 ml = sm.ml[x][row];
      if (!TWO) {
        const float2 mlA = sm.ml[0][row], mlB = sm.ml[1][row];
        const float mj = fmaxf(mlA.x, mlB.x);
        fA = ex2(mlA.x - mj);
        fB = ex2(mlB.x - mj);
        ml = make_float2(mj, mlA.y * fA + mlB.y * fB);
      }
      softmax_sync();
      const bool hasA = TWO ? x == 0 : cnt > 1 || ((j - 1) & 1) == 0, hasB = TWO ? x == 1 : cnt > 1 || ((j - 1) & 1) == 1;
      const bool starts = w.p == 0, ends = w.p + cnt == w.steps;
      const long long ub = u0 + (units - left) - w.p;
      const int c0 = (int)(ub / share), pieces = (int)((ub + w.steps - 1) / share) - c0 + 1;
      if (starts && ends) ml.y = 1.f / ml.y;
      sm.ml[x][row] = ml;
      constexpr int kTile = TWO ? 2 * kRows : kRows;
      auto write = [&](int r, int y, float4 v, float inv_sum) {
        const int rq = row_of(r);
        uint16_t* o = a.out + (int64_t)(w.s.r0 + row0 + rq) * a.out_stride + (size_t)(w.h * a.group + r - rq * a.group) * D + 4 * y;
        *(uint2*)o = make_uint2(f2bf(v.x * inv_sum) | (uint32_t)f2bf(v.y * inv_sum) << 16,
                                f2bf(v.z * inv_sum) | (uint32_t)f2bf(v.w * inv_sum) << 16);
      };
      // Half of the dims at a time through shared memory (the group's weights'
      // place), so that a row is written by neighbouring lanes: row r's 16-byte
      // word y stands at y ^ (r mod D / 8). Columns jd D/4 + y of O hold dim 4 y + jd.
      constexpr int kHalf = D / 8;
      float4* tile = (float4*)sm.p[x];
#pragma unroll 1
      for (int half = TWO ? 0 : x; half <= (TWO ? 1 : x) && active; ++half) {
#pragma unroll 1
        for (int y0 = 0; y0 < kHalf; y0 += 8) {
          float o[4][8];
#pragma unroll
          for (int jd = 0; jd < 4; ++jd) {
            uint32_t rA[8], rB[8];
            if (hasA) tmem_ld8(rA, to + jd * (D / 4) + half * kHalf + y0);
            if (hasB) tmem_ld8(rB, to + 128 + jd * (D / 4) + half * kHalf + y0);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              o[jd][e] = 0.f;
              if (hasA) o[jd][e] = __uint_as_float(rA[e]) * fA;
              if (hasB) o[jd][e] = fmaf(__uint_as_float(rB[e]), fB, o[jd][e]);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            tile[row * kHalf + ((y0 + e) ^ (row & (kHalf - 1)))] = make_float4(o[0][e], o[1][e], o[2][e], o[3][e]);
        }
        group_sync(x);
        constexpr int E = 4, kStep = 4 * (32 / kHalf);  // rows of a lane at once, rows of the group's warps
        const int y = lane % kHalf, last = min(kRows, cols - (TWO ? 128 * x : 0));
#pragma unroll 1
        for (int r1 = (warp & 3) * (32 / kHalf) + lane / kHalf; r1 < last; r1 += E * kStep) {
          float4 v[E];
          float2 m2[E];
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const int rl = (r1 + k * kStep) % kRows;
            v[k] = tile[rl * kHalf + (y ^ (rl & (kHalf - 1)))];
            m2[k] = sm.ml[x][rl];
          }
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const int rl = r1 + k * kStep, r = TWO ? 128 * x + rl : rl;
            if (rl >= last) continue;
            if (starts && ends) {
              write(r, half * kHalf + y, v[k], m2[k].y);
            } else {
              float* part = a.part + ((size_t)(2 * blockIdx.x + starts) * kTile + r) * kCol;
              *(float4*)(part + 4 * (half * kHalf + y)) = v[k];
              if (y == 0) *(float2*)(part + D) = m2[k];
            }
          }
        }
        group_sync(x);
      }
      if (!(starts && ends)) {
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
            auto partial = [&](int i) { return a.part + ((size_t)(2 * (c0 + i) + (i == 0)) * kTile + r) * kCol; };
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
            if (lane < D / 4) write(r, lane, v, 1.f / ss);
          }
        }
      }
      softmax_sync();  // this tile's maxima and sums have been read
      left -= cnt;
      w.p += cnt;
      if (w.p == w.steps) w.next_tile(a);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

static_assert(sizeof(ChunkSmem<128, true>) <= 227 * 1024 && sizeof(ChunkSmem<128, false>) <= 227 * 1024,
              "shared memory of a CTA");

template <int D, bool TWO>
cudaError_t launch_chunk(const ChunkArgs& a, int sms, cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(sms);
  lc.blockDim = dim3(kThreadsC);
  lc.dynamicSmemBytes = sizeof(ChunkSmem<D, TWO>);
  lc.stream = s;
  cudaLaunchAttribute at[1];
  early_launch(lc, at);
  return cudaLaunchKernelEx(&lc, chunk_kernel<D, TWO>, a);
}
template <int D, bool TWO>
cudaError_t setup_chunk() {
  return cudaFuncSetAttribute(chunk_kernel<D, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(ChunkSmem<D, TWO>));
}

}  // namespace

cudaError_t kv8_chunk_setup(int d) {
  cudaError_t e = d == 64 ? setup_chunk<64, false>() : setup_chunk<128, false>();
  if (e == cudaSuccess) e = d == 64 ? setup_chunk<64, true>() : setup_chunk<128, true>();
  return e;
}

size_t kv8_chunk_workspace(int d, int sms) { return 2 * (size_t)sms * 2 * kRows * (d + 4) * sizeof(float); }

bool kv8_chunk_fits(const Kv8View& v, const Kv8Batch& q, int group, long long pages) {
  const long long tiles = q.n_rows / (kRows / group) + q.B, steps = pages * kPage / kKeys + 2;
  return tiles * v.nkv < ((1ll << 31) - 4096) / steps;  // 4096: rounding up to shares
}

cudaError_t kv8_chunk(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                      int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, unsigned* arrived, float* part,
                      cudaStream_t s) {
  const bool two = (long long)q.n_rows * group * v.nkv >= 2ll * sms * 2 * kRows;
  ChunkArgs a{v, q, group, (two ? 2 : 1) * kRows / group, (65536 + group - 1) / group, qp, q_stride, std::fabs(scale) * kLog2e,
              scale < 0.f ? -1.f : 1.f, out, out_stride, part, arrived};
  if (d == 64) return two ? launch_chunk<64, true>(a, sms, s) : launch_chunk<64, false>(a, sms, s);
  return two ? launch_chunk<128, true>(a, sms, s) : launch_chunk<128, false>(a, sms, s);
}

}  // namespace qtts
