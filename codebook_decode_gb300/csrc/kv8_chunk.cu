// kv8_chunk.cu -- attention of many query rows over the 8-bit paged K/V cache,
// on the tcgen05 tensor cores (prompts, and batches with prompts among them).
//
// A tile is up to 128 or 256 rows (query tokens x the q heads of one kv head)
// of one session. For every 128 keys (8 pages)
//   S [128 x 128] = Q . K^T,   O [128 x d] += P . V
// with S, P and O in tensor memory (P takes the place of the scores it comes
// from) and Q, K and V as half in shared memory, K-major with the 128-byte
// swizzle. Codes are exact in half; the blocks' scales act outside the
// products, as in kv8_attention.cu: the K scale on the scores, the V scale on
// the weights.
//
// Warps: two softmax groups of four (a thread per row), four warps that widen a
// step's K codes into shared memory, four for its V codes, and one that issues
// the products. With 256 rows the groups have 128 each and a step's widened
// codes serve both; with 128 they take the steps in turn, each with its own S,
// P, O, maximum and sum, which are joined at the tile's end. Either way one
// group's softmax runs beside the other's products.
//
// Bound by the chain of a group's step (scores, maximum, weights, product: some
// 5500 cycles for two steps, against 2200 of their four products) and by what
// comes before and after: 1024 rows behind 1000 tokens, 16 q and 8 kv heads of
// 128, take 32 us (0.39 PFLOP/s), of which 6 us go before the first step and 3
// after the last; 30000 tokens back 332 us (0.77 PFLOP/s).
// What moved it most was code size and local memory: with the waits unrolled and
// each role's place in the work in registers the code had 165 KB, did not stay in
// the instruction cache, and spilled into a first-level cache of a few KB (40 us).
// What still spills at head_dim 128 are 40 bytes a thread (20 in the 256-row form).
//
// A weight leaves fp32's range, and the sum, where its block's V scale is not 0 but below
// 2^-100 of another one that counts in the same row.
//
// Work is cut into equal shares of key steps, one per CTA; tiles that several
// CTAs share are joined through the workspace by the last to arrive, in order.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv8.cuh"
#include "kv8_attn.cuh"
#include "tcgen05.cuh"

namespace qtts {
namespace {

constexpr int kRows = 128, kKeys = 128, kPagesPerStep = kKeys / kPage;
constexpr int kSoftmaxThreads = 256, kWidenThreads = 256;
constexpr int kThreadsC = kSoftmaxThreads + kWidenThreads + 128;
// registers of a thread: launched, then of the softmax, widening and issuing groups
constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsWiden = 72, kRegsIssue = 48;
static_assert(kSoftmaxThreads * kRegsSoftmax + kWidenThreads * kRegsWiden + 128 * kRegsIssue <= kThreadsC * kRegsLaunch,
              "the groups share what the block was launched with");
constexpr int kChunkTries = 1 << 17;  // bound of each wait; a try sleeps up to about 10 us
// What a cut tile costs beside its steps (queries prepared twice, partials out and in),
// in key steps: 6 and 12 measured the same, 3 and 0 cut calls that take 32 us whole into
// 44 us.
constexpr int kJoinSteps = 6;
// Pairs of pages unrolled in the passes for the maximum and for the weights, where no
// row is masked: 2 and 4 measured 32.4 us, 1 and 2 34.0, 4 and 4 33.0.
constexpr int kTurnsMax = 2, kTurnsWeights = 4;
constexpr int kIssueWarp = (kSoftmaxThreads + kWidenThreads) / 32;
constexpr int kPlaces = kWidenThreads / 32 + 2, kIssuePlace = kPlaces - 2, kSoftmaxPlace = kPlaces - 1;

// of the 16 columns (of k) number ks: their place in units of 16 bytes
__host__ __device__ constexpr uint64_t k_step(int ks, int rows) { return (ks / 4 * rows * 128 + ks % 4 * 32) / 16; }

struct ChunkArgs {
  Kv8View c;
  Kv8Batch q;
  int group, rows_per_tile, group_mul;  // r / group = r * group_mul >> 16 for r < 256
  const uint16_t* qp;
  int64_t q_stride;
  float scale_log2, q_sign;  // |softmax scale| log2 e, and its sign
  uint16_t* out;
  int64_t out_stride;
  float* part;        // [2 CTAs][D / 4][tile rows] float4, then [tile rows] maximum and sum (D + 4 floats a row)
  unsigned* arrived;  // [CTAs]
};

__device__ __forceinline__ int tile_steps(int L, int n, int t, int rows_per_tile) {
  return (L + min((t + 1) * rows_per_tile, n) + kKeys - 1) / kKeys;
}

// A place in the work: key step p of tile t of kv head h of session b. Each role
// keeps its own in shared memory: in registers it pushed others out to local
// memory, which misses the little first-level cache that is left.
struct Place {
  int b, h, t, p, steps;
  Kv8Session s;
  __device__ __forceinline__ void enter(const ChunkArgs& a, int bb) {
#pragma unroll 1
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
#pragma unroll 1
    while (p >= steps) {
      const int over = p - steps;
      next_tile(a);
      p = over;
    }
  }
};

template <int D, bool TWO>
struct ChunkSmem {
  alignas(1024) uint8_t q[TWO ? 2 : 1][kRows * D * 2];
  uint8_t out[kRows * D * 2 * (TWO ? 2 : 1)];  // results on their way out; before the first step the rows' query scales
  uint8_t k[2][kKeys * D * 2];
  uint8_t v[TWO ? 1 : 2][kKeys * D * 2];
  float2 ml[2][kRows];  // each group's maximum and sum
  // a page's K scale, logarithm of its V scale (for the maximum), and the V scale that its
  // weights are multiplied with: reciprocal and logarithm
  float4 sc[4][kPagesPerStep];
  // kfull, vfull: widened; kdone, vdone: read by the products; sdone: a group's
  // scores are there; pfull: its weights; pvdone: its second product has run;
  // qfull: the tile's queries; drained: all products have run
  uint64_t kfull[2], vfull[2], kdone[2], vdone[2], sdone[2], pfull[2], pvdone[2], qfull, drained;
  Place at[kPlaces];  // of the widening warps, the issuing warp and the softmax groups
  uint32_t tmem;
  int failed, verdict, flag, share, units;
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

// Loads into their registers or not: a choice after the load would wait for it.
__device__ __forceinline__ void load_if(uint4& v, const void* p, bool yes) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n @p ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "l"(p), "r"((uint32_t)yes));
}
__device__ __forceinline__ void load_if(float2& v, const void* p, bool yes) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %3, 0;\n @p ld.global.v2.f32 {%0,%1}, [%2];\n}"
               : "+f"(v.x), "+f"(v.y)
               : "l"(p), "r"((uint32_t)yes));
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
template <int R>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ uint32_t bf2_bits(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *(const uint32_t*)&p;
}
// largest finite halves for what is above them: weights of blocks of zeros
__device__ __forceinline__ uint32_t half2_finite(float a, float b) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
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
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// A from tensor memory: a row's halves two to a column
__device__ __forceinline__ void tc_mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
    int u0 = 0, u1 = 0;
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
        } else if (lo <= u0 && u0 < lo + own) {
          const int at = u0 - lo, h = at / per;
          int sum;
          Place& w = sm.at[0];
          w.b = b0 + lane;
          w.h = h;
          w.t = tiles_until(ses, a.rows_per_tile, whole, at - h * per, sum);
          w.p = at - h * per - sum;
          w.steps = tile_steps(ses.L, ses.n, w.t, a.rows_per_tile);
          w.s = ses;
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
        const int each = tiles / G, more = tiles - each * G, me = blockIdx.x;
        whole = (long long)(each + (more > 0)) * most <= share + kJoinSteps;
        u0 = whole ? me * each + min(me, more) : me * share;
        u1 = whole ? u0 + each + (me < more) : min(u0 + share, total);
        if (u0 >= u1) break;
      }
    }
    // key steps of this CTA
    __syncwarp();
    const Place first = sm.at[0];
    int units = max(u1 - u0, 0);
    if (whole && units) {
      Place x = first;
      const int count = units;
      units = x.steps;
#pragma unroll 1
      for (int i = 1; i < count; ++i) {
        x.next_tile(a);
        units += x.steps;
      }
    }
    if (lane > 0 && lane < kPlaces) sm.at[lane] = first;
    if (lane == 0) {
      sm.share = share;
      sm.units = units;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int units = sm.units;
  // Bounded; once one wait has run out all others give up too. Short: it is in many places.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
#pragma unroll 1
    for (int tries = 0; tries < kChunkTries && !*(volatile int*)&sm.failed; ++tries)
      if (mbar_test_sleep(bar, parity, 10000)) return true;
    *(volatile int*)&sm.failed = 1;
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
    int j;
    bool ok = true;
    // lane x holds the block of page x & 1 of this warp's two, of step 16 k + x / 2
    // (-1: beyond the tile); the next 16 steps' are fetched meanwhile
    Place& ahead = sm.at[warp - kSoftmaxThreads / 32];
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
      __syncwarp();
      if (lane == 0 && 16 * (k + 1) < units) {
        Place x = ahead;
        x.advance(a, 16);
        ahead = x;
      }
      __syncwarp();
      return id;
    };
    int ids = -1, ids_next = -1;
    const int left = units;
    // K: a lane of a load is one of 8 tokens x 4 words. V: lane x takes the 4 dims
    // 4x.. (d = 64: of half the words)
    constexpr int D4 = D / 4, kWords = D / 32;  // 16-byte words of a lane and page
    const int r8 = lane & 7, dch = lane >> 3, x4 = lane % D4;
    const size_t lane_at = is_v ? 16 * D + x4 * 64 + (D == 128 ? 0 : lane / D4 * 32) : dch * 16;
    uint4 wd[2][kWords];
    float2 sc[2];
    auto load = [&](int step) {
      const uint4 none = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);  // codes of 0
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int id = __shfl_sync(0xffffffffu, ids, 2 * (step & 15) + i);
        const uint8_t* src = a.c.codes + (size_t)max(id, 0) * (32 * D) + lane_at;
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const int at = is_v ? e * 16 : e % (D / 64) * 1024 + token_of(e / (D / 64) * 8 + r8) * 64;
          wd[i][e] = none;
          load_if(wd[i][e], src + at, id >= 0);
        }
        sc[i] = make_float2(0.f, 0.f);
        load_if(sc[i], a.c.scales + 2 * (size_t)max(id, 0), !is_v && id >= 0);
      }
    };
    // step -1 only asks for the first step's codes
#pragma unroll 1
    for (j = -1; j < left; ++j) {
      if (j >= 0) {
        const int s = j & 1;
        if (!is_v) {
          if (j >= 2) ok = wait(&sm.kdone[s], ((j >> 1) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane < 2) {
            const float2 v = lane ? sc[1] : sc[0];
            // A block of zeros moves no maximum, and its weights, multiplied with nothing but
            // zeros, are only summed: as they are, since 2^-100 of them may be below fp32's range.
            const float sv = v.y != v.y ? v.y : fmaxf(v.y, kKv8MinScale), lv = lg2(sv);
            sm.sc[j & 3][wp + lane] = make_float4(v.x, lv, v.y == 0.f ? 1.f : 1.f / sv, v.y == 0.f ? 0.f : lv);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
              const uint4 k = wd[i][e];
              uint8_t* dst = sm.k[s] + e % (D / 64) * (kKeys * 128);
              const int row = (wp + i) * kPage + e / (D / 64) * 8 + r8;
              uint4 lo, hi;
              widen(k.x, lo.x, lo.y);
              widen(k.y, lo.z, lo.w);
              widen(k.z, hi.x, hi.y);
              widen(k.w, hi.z, hi.w);
              *(uint4*)(dst + word_at(row, 2 * dch)) = lo;
              *(uint4*)(dst + word_at(row, 2 * dch + 1)) = hi;
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
      }
      if (j < 0 || (j & 15) == 8) {
        ids_next = fetch_ids((j + 8) >> 4);
        if (j < 0) ids = ids_next;
      }
      if ((j & 15) == 15 && j > 0) ids = ids_next;
      if (j + 1 < left) load(j + 1);
    }
  } else if (warp >= kIssueWarp) {
    // ---- products
    set_regs_down<kRegsIssue>();
    if (warp == kIssueWarp) {
      // The whole warp goes through the loop, so that descriptors stay in uniform
      // registers; one lane, always the same, issues.
      const bool leader = elect_one();
      constexpr uint32_t idS = idesc_f16(kRows, kKeys), idO = idesc_f16(kRows, D);
      int j = 0, seg = 0, left = units;
      uint32_t odd = 0;  // bit x: group x has had an odd number of steps
      bool ok = true;
      auto scores = [&](int jj, int x, bool last) {  // group x's scores of step jj; last: K's place is free after
        const int s = jj & 1;
        ok = __all_sync(0xffffffffu, wait(&sm.kfull[s], (jj >> 1) & 1));
        if (!ok) return;
        tc_fence_after();
        // a descriptor's low bits are the address in 16-byte units: steps along k add to it
        const uint64_t qd = swizzled_desc(sm.q[TWO ? x : 0]), kd = swizzled_desc(sm.k[s]);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma(tmem + 128 * x, qd + k_step(ks, kRows), kd + k_step(ks, kKeys), idS, ks > 0);
          tc_commit(&sm.sdone[x]);
          mbar_arrive(&sm.sdone[x]);
          if (last) tc_commit(&sm.kdone[s]);
        }
        __syncwarp();
      };
      auto weights_there = [&](int x) {  // group x has read its scores and written its weights
        ok = __all_sync(0xffffffffu, wait(&sm.pfull[x], odd >> x & 1));
        odd ^= 1u << x;
        return ok;
      };
      auto values = [&](int jj, int x, bool first, bool last) {  // group x's second product of step jj
        const int vs = TWO ? 0 : jj & 1;
        ok = __all_sync(0xffffffffu, wait(&sm.vfull[vs], TWO ? jj & 1 : (jj >> 1) & 1));
        if (!ok) return;
        tc_fence_after();
        const uint64_t vd = swizzled_desc(sm.v[vs]);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            tc_mma_tmem(tmem + 256 + 128 * x, tmem + 128 * x + 8 * ks, vd + k_step(ks, D), idO, !first || ks > 0);
          tc_commit(&sm.pvdone[x]);
          if (last) tc_commit(&sm.vdone[vs]);
        }
        __syncwarp();
      };
      // A group's next scores land where its weights stood: the product that reads
      // those has to have run (products on different accumulators may pass each other).
      auto weights_read = [&](int x) { return ok = __all_sync(0xffffffffu, wait(&sm.pvdone[x], (odd >> x & 1) ^ 1)); };
#pragma unroll 1
      while (left && ok) {
        const Place& w = sm.at[kIssuePlace];
        const int cnt = min(left, w.steps - w.p), j0 = j, j1 = j + cnt;
        ok = __all_sync(0xffffffffu, wait(&sm.qfull, seg & 1));
        tc_fence_after();
        if constexpr (TWO) {
          const bool both = min(a.rows_per_tile, w.s.n - w.t * a.rows_per_tile) * a.group > kRows;
#pragma unroll 1
          for (int x = 0; x <= both && ok; ++x) scores(j, x, x == both);
#pragma unroll 1
          for (; j < j1 && ok; ++j)
#pragma unroll 1
            for (int x = 0; x <= both && ok; ++x) {
              if (weights_there(x)) values(j, x, j == j0, x == both);
              if (ok && j + 1 < j1 && weights_read(x)) scores(j + 1, x, x == both);
            }
        } else {
#pragma unroll 1
          for (int i = 0; i < min(cnt, 2) && ok; ++i) scores(j + i, (j + i) & 1, true);
#pragma unroll 1
          for (; j < j1 && ok; ++j) {
            if (weights_there(j & 1)) values(j, j & 1, j - j0 < 2, true);
            if (ok && j + 2 < j1 && weights_read(j & 1)) scores(j + 2, j & 1, true);
          }
        }
        left -= cnt;
        ++seg;
        __syncwarp();
        if (leader && left) sm.at[kIssuePlace].advance(a, cnt);
        __syncwarp();
      }
      drain_products(&sm.drained, kChunkTries);
    }
    __syncwarp();
  } else {
    // ---- softmax: thread = row; group x has its own rows, or takes the steps of its parity
    set_regs_up<kRegsSoftmax>();
    const int x = warp >> 2, row = tid & 127;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + 128 * x + quarter, to = tmem + 256 + quarter;
    int j = 0, left = units;
    uint32_t odd = 0;  // this group has had an odd number of steps
    bool ok = true;
    const Place& w = sm.at[kSoftmaxPlace];
    // The rows' query scales stand in the results' place: that is next written behind
    // two barriers of both groups. A place that one group writes when its steps are done
    // would not do: a group without a step in this tile comes there while the other still
    // reads its scales.
    float* query_scale = (float*)sm.out;
#pragma unroll 1
    while (left && ok) {
      const int cnt = min(left, w.steps - w.p);
      const int row0 = w.t * a.rows_per_tile, rows = min(a.rows_per_tile, w.s.n - row0), cols = rows * a.group;
      const bool active = !TWO || x == 0 || cols > kRows;
      // The tile's queries, rotated, into shared memory: four lanes a row, each with
      // every fourth 4 dims and their partners D/2 further. Scaled by the power of
      // two of the row's largest magnitude (before the rotation, which can grow it
      // by sqrt 2: half has room).
      constexpr int kQuads = D / 32;  // of a lane
#pragma unroll 1
      for (int r = tid / 4; r - tid / 4 < cols; r += kSoftmaxThreads / 4) {
        const int rc = min(r, cols - 1), rq = row_of(rc), at = tid % 4 * 4;
        const uint16_t* src = a.qp + (int64_t)(w.s.r0 + row0 + rq) * a.q_stride + (size_t)(w.h * a.group + rc - rq * a.group) * D + at;
        const size_t turn = (size_t)(w.s.L + row0 + rq) * (D / 2) + at;
        uint2 lo[kQuads], hi[kQuads];
        ulonglong2 cs[kQuads];
        float4 sn[kQuads];
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          lo[k] = *(const uint2*)(src + 16 * k);
          hi[k] = *(const uint2*)(src + 16 * k + D / 2);
          if (a.c.rope_cos) {
            cs[k] = *(const ulonglong2*)(a.c.rope_cos + turn + 16 * k);
            sn[k] = *(const float4*)(a.c.rope_sin + turn + 16 * k);
          }
        }
        uint32_t mag = 0;
#pragma unroll
        for (int k = 0; k < kQuads; ++k)
          mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(lo[k].x & 0x7fff7fffu, lo[k].y & 0x7fff7fffu),
                                       __vmaxu2(hi[k].x & 0x7fff7fffu, hi[k].y & 0x7fff7fffu)));
        mag = __vmaxu2(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
        mag = __vmaxu2(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
        mag = max(mag & 0xffffu, mag >> 16);
        const uint32_t ex = min(max(mag << 16 & 0x7f800000u, 1u << 23), 253u << 23);
        const float inv = __uint_as_float((254u << 23) - ex) * a.q_sign;
        if (r < cols && at == 0) query_scale[r] = __uint_as_float(ex) * a.scale_log2;
        uint8_t* dst = sm.q[TWO ? r >> 7 : 0] + (at & 4) * 2;
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          uint64_t p0 = pack2(__uint_as_float(lo[k].x << 16) * inv, __uint_as_float(lo[k].x & 0xffff0000u) * inv);
          uint64_t p1 = pack2(__uint_as_float(lo[k].y << 16) * inv, __uint_as_float(lo[k].y & 0xffff0000u) * inv);
          uint64_t q0 = pack2(__uint_as_float(hi[k].x << 16) * inv, __uint_as_float(hi[k].x & 0xffff0000u) * inv);
          uint64_t q1 = pack2(__uint_as_float(hi[k].y << 16) * inv, __uint_as_float(hi[k].y & 0xffff0000u) * inv);
          if (a.c.rope_cos) {
            const uint64_t s0 = pack2(sn[k].x, sn[k].y), s1 = pack2(sn[k].z, sn[k].w);
            const uint64_t m0 = pack2(-sn[k].x, -sn[k].y), m1 = pack2(-sn[k].z, -sn[k].w);
            const uint64_t u0 = p0, u1 = p1;
            p0 = fma2(u0, cs[k].x, mul2(q0, m0));
            p1 = fma2(u1, cs[k].y, mul2(q1, m1));
            q0 = fma2(q0, cs[k].x, mul2(u0, s0));
            q1 = fma2(q1, cs[k].y, mul2(u1, s1));
          }
          const float2 y0 = unpack2(p0), y1 = unpack2(p1), z0 = unpack2(q0), z1 = unpack2(q1);
          if (r < cols) {  // dims 16 k + at.. and D / 2 + 16 k + at..
            const int word = 2 * k + at / 8;
            *(uint2*)(dst + word_at(r & 127, word)) = make_uint2(half2_bits(y0.x, y0.y), half2_bits(y1.x, y1.y));
            *(uint2*)(dst + (D == 128 ? kRows * 128 + word_at(r & 127, word) : word_at(r & 127, 4 + word))) =
                make_uint2(half2_bits(z0.x, z0.y), half2_bits(z1.x, z1.y));
          }
        }
      }
      softmax_sync();
      const int tile_row = TWO ? 128 * x + row : row;
      const float cf = tile_row < cols ? query_scale[tile_row] : 0.f;
      fence_async_shared();
      tc_fence_before();  // the last tile's accumulators have been read
      mbar_arrive(&sm.qfull);

      float m = kNone, l = 0.f;
      bool any = false;  // steps of this group in this tile
      // of the tile's keys from this CTA's first step on: the last that this row
      // sees, and the step from which on a row does not see all
      int lim = w.s.L + row0 + min(row_of(TWO ? 128 * x + row : row), rows - 1) - w.p * kKeys;
      const int first_masked = j + (w.s.L + row0 + 1) / kKeys - w.p;
#pragma unroll 1
      for (const int end = j + cnt; j < end && ok; ++j, lim -= kKeys) {
        if (TWO ? !active : (j & 1) != x) continue;
        ok = __all_sync(0xffffffffu, wait(&sm.sdone[x], odd));
        if (!ok) break;
        tc_fence_after();
        const float4* sc = sm.sc[j & 3];
        // One path for steps that every row sees whole and one for the others: the
        // first without jumps (each costs an instruction fetch).
        auto work = [&](auto masked) {
          constexpr bool kMasked = decltype(masked)::value;
          // The scores come a page at a time, the next page's load beside the work on
          // this one: first from the last page down, for the maximum, then up again.
          // Two pages a turn: unrolled in full, the roles' code outgrew the instruction
          // cache.
          uint32_t r0[16], r1[16];
          auto load = [&](uint32_t (&v)[16], int page) { tmem_ld16(v, ts + 16 * page); };
          auto mask = [&](uint32_t (&v)[16], int page) {
            if constexpr (kMasked) {
#pragma unroll
              for (int n = 0; n < 16; ++n)
                if (page * kPage + token_of(n) > lim) v[n] = 0xff800000u;  // -inf
            }
          };
          // a page's factors: of one that the row does not see at all they are
          // harmless ones, whatever its scales
          auto factors = [&](int page) {
            float4 f = sc[page];
            if (kMasked && page * kPage > lim) f = make_float4(1.f, 0.f, 1.f, 0.f);
            f.x = max_nan(f.x * cf, kKv8MinScale);  // positive: -inf stays -inf
            return f;
          };
          float mx = kNone;
          auto top = [&](uint32_t (&v)[16], int page) {
            mask(v, page);
            auto at = [&](int e) { return __uint_as_float(v[e]); };
            float g = max3(at(0), at(1), at(2));
#pragma unroll
            for (int e = 3; e < 15; e += 2) g = max3(g, at(e), at(e + 1));
            g = fmaxf(g, at(15));
            const float4 f = factors(page);
            mx = fmaxf(mx, fmaf(g, f.x, f.y));
          };
          load(r1, kPagesPerStep - 1);
#pragma unroll(kMasked ? 1 : kTurnsMax)
          for (int page = kPagesPerStep - 2; page >= 0; page -= 2) {
            tmem_wait_ld(r1);
            load(r0, page);
            top(r1, page + 1);
            tmem_wait_ld(r0);
            if (page) load(r1, page - 1);
            top(r0, page);
          }
          const bool grow = mx > m + kSlack;
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
            const float f = grow ? ex2(m - mx) : 1.f;
            if (grow) {
              l = rebase(l, m, mx);
              m = mx;
            }
            if (any) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(o, to + 128 * x + 16 * c);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(to + 128 * x + 16 * c, o);
              }
              tmem_wait_st();
            }
          }
          // They take the place of scores that this thread has read: a page's 16 halves
          // 8 columns from 8 page on.
          auto weights = [&](uint32_t (&v)[16], int page) {
            const float4 f = factors(page);
            const uint64_t mul = pack2(f.x, f.x), off = pack2(f.w - m, f.w - m);
            uint64_t sum = 0;
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 y = unpack2(fma2(pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), mul, off));
              const float p0 = ex2(y.x), p1 = ex2(y.y);  // weight times V scale
              sum = add2(sum, pack2(p0, p1));
              h[e] = half2_finite(p0, p1);
            }
            const float2 t = unpack2(sum);
            l = fmaf(t.x + t.y, f.z, l);
            tmem_st8(ts + 8 * page, h);
          };
#pragma unroll(kMasked ? 1 : kTurnsWeights)
          for (int page = 0; page < kPagesPerStep; page += 2) {
            if (page) {
              tmem_wait_ld(r0);
              mask(r0, page);
            }
            load(r1, page + 1);
            weights(r0, page);
            tmem_wait_ld(r1);
            if (page + 2 < kPagesPerStep) load(r0, page + 2);
            mask(r1, page + 1);
            weights(r1, page + 1);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sm.pfull[x]);
          any = true;
          odd ^= 1;
        };
        if (j >= first_masked) work(std::true_type{});
        else work(std::false_type{});
      }
      if (ok && any) ok = wait(&sm.pvdone[x], odd ^ 1);  // the group's last product
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
        ml = make_float2(mj, rebase(mlA.y, mlA.x, mj) + rebase(mlB.y, mlB.x, mj));
      }
      const bool hasA = TWO ? x == 0 : cnt > 1 || ((j - 1) & 1) == 0, hasB = TWO ? x == 1 : cnt > 1 || ((j - 1) & 1) == 1;
      const bool starts = w.p == 0, ends = w.p + cnt == w.steps;
      const bool closed = starts && ends;
      // Columns jd D/4 + y of O hold dim 4 y + jd: a thread takes 16 dims of its row at
      // a time (groups on the same rows: half of the dims each). Results go through
      // shared memory as bf16 (row r's 16-byte word y at y ^ (r mod D / 8)), so that a
      // row is written by neighbouring lanes; a shared tile's partials straight to the
      // workspace, there [16-byte words][rows].
      constexpr int kTile = TWO ? 2 * kRows : kRows, kWords = D / 8;
      const int mine = TWO ? 128 * x + row : row;  // the thread's row of the tile
      const int at0 = TWO ? 0 : x * (D / 32), at1 = TWO ? D / 16 : at0 + D / 32;
      auto put = [&](int r, int at, const float4 (&v)[4], float f) {
        uint8_t* dst = sm.out + r * (2 * D);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *(uint4*)(dst + (((2 * at + e) ^ (r & (kWords - 1))) << 4)) =
              make_uint4(bf2_bits(v[2 * e].x * f, v[2 * e].y * f), bf2_bits(v[2 * e].z * f, v[2 * e].w * f),
                         bf2_bits(v[2 * e + 1].x * f, v[2 * e + 1].y * f), bf2_bits(v[2 * e + 1].z * f, v[2 * e + 1].w * f));
      };
      auto partial = [&](int slot) { return (float4*)(a.part + (size_t)slot * kTile * kCol); };
      float4* part = partial(2 * blockIdx.x + starts);
      const float inv_sum = 1.f / ml.y;
#pragma unroll 1
      for (int at = at0; at < at1 && active; ++at) {
        uint32_t rA[4][4], rB[4][4];
#pragma unroll
        for (int jd = 0; jd < 4; ++jd) {
          if (hasA) tmem_ld4(rA[jd], to + jd * (D / 4) + 4 * at);
          if (hasB) tmem_ld4(rB[jd], to + 128 + jd * (D / 4) + 4 * at);
        }
        tmem_wait_ld();
        float4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float o[4];
#pragma unroll
          for (int jd = 0; jd < 4; ++jd) {
            o[jd] = 0.f;
            if (hasA) o[jd] = __uint_as_float(rA[jd][e]) * fA;
            if (hasB) o[jd] = fmaf(__uint_as_float(rB[jd][e]), fB, o[jd]);
          }
          v[e] = make_float4(o[0], o[1], o[2], o[3]);
        }
        if (closed) {
          put(mine, at, v, inv_sum);
        } else if (mine < cols) {
#pragma unroll
          for (int e = 0; e < 4; ++e) part[(4 * at + e) * kTile + mine] = v[e];
          if (at == 0) ((float2*)(part + D / 4 * kTile))[mine] = ml;
        }
      }
      bool write = true;
      if (!closed) {
        // the tile's first key step, the CTA that has it, and the number of CTAs on the tile
        const int share = sm.share, ub = blockIdx.x * share + (units - left) - w.p;
        const int c0 = ub / share, pieces = (ub + w.steps - 1) / share - c0 + 1;
        __threadfence();
        softmax_sync();
        if (tid == 0) {
          sm.flag = atomicAdd(&a.arrived[c0], 1u) == (unsigned)pieces - 1;
          if (sm.flag) a.arrived[c0] = 0;  // ready for the next call
        }
        softmax_sync();
        write = sm.flag;
        if (write) {  // the last to arrive joins the tile's partials, in their order
          __threadfence();
          auto of = [&](int i) { return partial(2 * (c0 + i) + (i == 0)); };
#pragma unroll 1
          for (int item = tid; item < cols * (D / 16); item += kSoftmaxThreads) {
            const int at = item / cols, r = item - at * cols;
            auto sums = [&](int i) { return __ldcg((const float2*)(of(i) + D / 4 * kTile) + r); };
            float mj = kNone, sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) mj = fmaxf(mj, sums(i).x);
            float4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int i = 0; i < pieces; ++i) {
              const float2 y = sums(i);
              const float f = ex2(y.x - mj);
              sum += rebase(y.y, y.x, mj);
#pragma unroll
              for (int e = 0; e < 4; ++e) axpy(v[e], __ldcg(of(i) + (4 * at + e) * kTile + r), f);
            }
            put(r, at, v, 1.f / sum);
          }
        }
      }
      softmax_sync();
      if (write) {
        constexpr int kLanes = D / 4, kOnce = kSoftmaxThreads / kLanes;  // lanes of a row, rows at once
        const int y = tid % kLanes;
#pragma unroll 4
        for (int r = tid / kLanes; r < cols; r += kOnce) {
          const int rq = row_of(r);
          uint16_t* o = a.out + (int64_t)(w.s.r0 + row0 + rq) * a.out_stride + (size_t)(w.h * a.group + r - rq * a.group) * D + 4 * y;
          *(uint2*)o = *(const uint2*)(sm.out + r * (2 * D) + (((y >> 1) ^ (r & (kWords - 1))) << 4) + (y & 1) * 8);
        }
      }
      softmax_sync();  // this tile's maxima and sums have been read
      left -= cnt;
      if (tid == 0 && left) sm.at[kSoftmaxPlace].advance(a, cnt);
      softmax_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sm.failed) set_err(a.c.err, QTTS_DEV_TIMEOUT);
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

// Rows that the call's sessions can have: n_rows and max_new are bounds of any size.
static long long most_rows(const Kv8View& v, const Kv8Batch& q) {
  return std::min((long long)q.n_rows, (long long)q.B * std::min(q.max_new, v.max_context));
}

bool kv8_chunk_fits(const Kv8View& v, const Kv8Batch& q, int group, long long pages) {
  const long long tiles = most_rows(v, q) / (kRows / group) + q.B, steps = pages * kPage / kKeys + 2;
  return tiles * v.nkv < ((1ll << 31) - 4096) / steps;  // 4096: rounding up to shares
}

cudaError_t kv8_chunk(const Kv8View& v, const Kv8Batch& q, int d, int group, int sms, const uint16_t* qp,
                      int64_t q_stride, float scale, uint16_t* out, int64_t out_stride, unsigned* arrived, float* part,
                      cudaStream_t s) {
  const bool two = most_rows(v, q) * group * v.nkv >= 2ll * sms * 2 * kRows;
  ChunkArgs a{v, q, group, (two ? 2 : 1) * kRows / group, (65536 + group - 1) / group, qp, q_stride, std::fabs(scale) * kLog2e,
              scale < 0.f ? -1.f : 1.f, out, out_stride, part, arrived};
  if (d == 64) return two ? launch_chunk<64, true>(a, sms, s) : launch_chunk<64, false>(a, sms, s);
  return two ? launch_chunk<128, true>(a, sms, s) : launch_chunk<128, false>(a, sms, s);
}

}  // namespace qtts
