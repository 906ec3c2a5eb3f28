// w4_linear.cu -- products of up to 64 activation rows with 4-bit weights:
// y[m][n] = sum_k x[m][k] * code[n][k] * scale[n][k / group].
//
// Few rows are bound by the launch and one round of loads (one row, 4096 x 2048: 3.7 us;
// 12288 x 2048 in groups of 32 6.1 us, 2.3 TB/s), large layers by short CTAs that come in
// waves, each copying the activations before its first product (four rows, 30000 x 4096:
// 938 CTAs in 456 places, 32 us, 2.0 TB/s), not by the weights' bytes. The weights are
// the A operand of mma.sync m16n8k16 (16 output columns of the layer per
// tile), the activations the B operand (8 rows per n-tile), so that one
// activation row pads to 8, not to 16 or 128. Codes are exact in bf16 and are
// widened in registers (4 bits under the exponent of 2^7, minus 136); a
// group's scale multiplies its fp32 partial sums, so nothing is rounded before
// the result.
//
// Weights in memory: tiles of 16 rows x 64 k, one lane's 32 codes together
// (512 contiguous bytes a tile, tiles of a row block in k order): word e of
// lane (g, t) holds for rows g and g + 8 the codes of
//   k = 32 (e / 2) + 8 t + 4 (e % 2) + 0..3
// as the nibbles of one MMA's four A registers. Every MMA so lies inside 32
// consecutive k and one group, and a lane's activations are 16 contiguous
// bytes. Scales follow the same order: [row block][k tile][g][row half, 32-k
// half] for groups of 32, [row block][group][g][row half] above.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "device_util.cuh"
#include "qtts_internal.h"
#include "tcgen05.cuh"

struct qtts_w4 {
  int N = 0, K = 0, group = 0, device = 0, G = 0;
  int RB = 0, KT = 0;  // row blocks of 16, k tiles of 64
  qtts::ErrorText err;
  uint4* codes = nullptr;      // [RB][KT][32 lanes]
  uint16_t* scales = nullptr;  // [RB][units][16 or 32]
  bool loaded = false;
};

namespace qtts {
namespace {

namespace cg = cooperative_groups;

constexpr int kW4Rows = 16, kW4K = 64, kW4MaxM = 64;
constexpr int kW4Warps = 8, kW4Threads = 32 * kW4Warps;
constexpr int kW4MaxSplit = 4;  // CTAs of a cluster; clusters of 8 left SMs of a GPC unused and ran in two waves

// scales of one row block and k tile of 64 (groups of 32), or of one group
__host__ __device__ __forceinline__ int scale_units(int KT, int K, int group) { return group == 32 ? KT : K / group; }
// place of (row r of the block, 32-k half or 0) within its unit
__device__ __forceinline__ int scale_slot(int r, int half, int group) {
  return group == 32 ? (r & 7) * 4 + (r >> 3) * 2 + half : (r & 7) * 2 + (r >> 3);
}
__device__ __forceinline__ size_t scale_at(int n, int grp, int KT, int K, int group) {
  const int units = scale_units(KT, K, group);
  const size_t rb = n / kW4Rows;
  return group == 32 ? (rb * units + grp / 2) * 32 + scale_slot(n % kW4Rows, grp & 1, group)
                     : (rb * units + grp) * 16 + scale_slot(n % kW4Rows, 0, group);
}
// k of nibble j (0..3) of MMA e of a tile, for lane quad position t
__device__ __forceinline__ int k_of(int e, int t, int j) { return 32 * (e >> 1) + 8 * t + 4 * (e & 1) + j; }

// ---- load time: quantise, pack, unpack (natural order [N][K], [N][K / group])

__global__ void w4_quantize_kernel(const uint16_t* w, int N, int K, int group, int8_t* q, uint16_t* s) {
  const int groups = K / group, lane = threadIdx.x & 31;
  const long long total = (long long)N * groups;
  for (long long i = blockIdx.x * (blockDim.x / 32ll) + threadIdx.x / 32; i < total;
       i += gridDim.x * (blockDim.x / 32ll)) {
    const uint16_t* src = w + i * group;
    uint32_t mx = 0;
    for (int k = lane; k < group; k += 32) mx = max(mx, (uint32_t)src[k] & 0x7fffu);
    mx = __reduce_max_sync(0xffffffffu, mx);
    uint16_t sb = mx >= 0x7f80u ? (uint16_t)0x7fffu : f2bf(bf2f(mx) / 7.f);
    if (sb < 0x0080u) sb = 0;  // below the normal numbers
    const float sc = bf2f(sb);
    for (int k = lane; k < group; k += 32) {
      const float x = sb ? bf2f(src[k]) / sc : 0.f;
      q[i * group + k] = (int8_t)__float2int_rn(fminf(fmaxf(x, -7.f), 7.f));
    }
    if (lane == 0) s[i] = sb;
  }
}

__global__ void w4_pack_kernel(const int8_t* q, const uint16_t* s, int N, int K, int group, int RB, int KT,
                               uint4* codes, uint16_t* scales, int* bad) {
  const long long total = (long long)RB * KT * 32;
  const int groups = K / group;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += gridDim.x * (long long)blockDim.x) {
    const int lane = i & 31, g = lane >> 2, t = lane & 3;
    const int kt = (int)(i / 32 % KT), rb = (int)(i / 32 / KT);
    uint32_t w[4];
    for (int e = 0; e < 4; ++e) {
      w[e] = 0;
      for (int a = 0; a < 4; ++a)  // A register a: row g or g + 8, nibbles 2 (a / 2), 2 (a / 2) + 1
        for (int h = 0; h < 2; ++h) {
          const int n = rb * kW4Rows + g + 8 * (a & 1), k = kt * kW4K + k_of(e, t, 2 * (a >> 1) + h);
          int c = 0;
          if (n < N && k < K) c = q[(size_t)n * K + k];
          if (c < -8 || c > 7) *bad = 1;
          w[e] |= (uint32_t)((c + 8) & 15) << (4 * a + 16 * h);
        }
    }
    codes[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const long long ns = (long long)N * groups;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < ns; i += gridDim.x * (long long)blockDim.x)
    scales[scale_at((int)(i / groups), (int)(i % groups), KT, K, group)] = s[i];
}

__global__ void w4_unpack_kernel(const uint4* codes, const uint16_t* scales, int N, int K, int group, int KT,
                                 int8_t* q, uint16_t* s) {
  const long long total = (long long)N * K;
  const int groups = K / group;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += gridDim.x * (long long)blockDim.x) {
    const int n = (int)(i / K), k = (int)(i % K);
    const int r = n % kW4Rows, kk = k % kW4K;
    const int e = (kk >> 5) * 2 + ((kk >> 2) & 1), t = (kk >> 3) & 3, j = kk & 3;
    const uint4 v = codes[((size_t)(n / kW4Rows) * KT + k / kW4K) * 32 + (r & 7) * 4 + t];
    const uint32_t w = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
    const int a = (r >> 3) + 2 * (j >> 1);
    q[i] = (int8_t)((int)(w >> (4 * a + 16 * (j & 1)) & 15u) - 8);
  }
  const long long ns = (long long)N * groups;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < ns; i += gridDim.x * (long long)blockDim.x)
    s[i] = scales[scale_at((int)(i / groups), (int)(i % groups), KT, K, group)];
}

// ---- the product

struct W4Args {
  const uint4* codes;
  const uint16_t* scales;
  int N, K, RB, KT, group, sunits;
  int M;
  const uint16_t* x;
  int64_t x_stride;
  void* y;
  int64_t y_stride;
  int y_f32;
  int rw_log, s_log;  // 2^rw_log warps along the row blocks, the others along k; clusters of 2^s_log CTAs
  int chunk;  // k tiles of activations in shared memory at a time
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Two codes to a bf16 pair: 4 bits under the exponent of 2^7 are 128 + code +
// 8, minus 136 the code itself, exactly.
__device__ __forceinline__ uint32_t widen4(uint32_t w) {
  uint32_t r;
  const uint32_t off = 0x43084308u;  // 136, 136
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((w & 0x000f000fu) | 0x43004300u), "r"(off));
  return r;
}
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Loads that stay where they are written, ahead of their use.
__device__ __forceinline__ uint2 load_early8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_early4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// A CTA's warps stand rw along the row blocks (R blocks each) and 8 / rw along
// k, and the CTAs of a cluster split k further; partial sums meet in shared
// memory, across the cluster through distributed shared memory. The CTA's
// range of the activations is copied to shared memory (all rows, `chunk` k
// tiles at a time) while the first weights are on their way; without it every
// k tile waited for its activations.
template <int NT, int R>
__global__ void __launch_bounds__(kW4Threads, NT == 1 ? 3 : NT <= 4 ? 2 : 1) w4_kernel(const __grid_constant__ W4Args a) {
  extern __shared__ __align__(16) uint8_t w4_smem[];  // activations, then the sums [k warps][8 NT][rows + 4]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = 1 << a.s_log, rank = blockIdx.x & (S - 1), cta = blockIdx.x >> a.s_log;
  const int rw = 1 << a.rw_log, kw_log = 3 - a.rw_log, kw = 1 << kw_log, wr = warp & (rw - 1), wk = warp >> a.rw_log;
  const int cta_rows = 16 * R << a.rw_log, stride = cta_rows + 4;
  const int rb0 = ((cta << a.rw_log) + wr) * R;
  const int t0 = a.KT * rank >> a.s_log, t1 = a.KT * (rank + 1) >> a.s_log;
  const bool fine = a.group == 32;
  const int unit_log = a.group == 128 ? 1 : 0;  // k tiles of a unit of scales
  const uint4* codes = a.codes + (size_t)rb0 * a.KT * 32 + lane;
  const uint16_t* scales = a.scales + (fine ? (size_t)rb0 * a.sunits * 32 + 4 * g : (size_t)rb0 * a.sunits * 16 + 2 * g);
  const size_t codes_step = (size_t)a.KT * 32, scales_step = (size_t)a.sunits * (fine ? 32 : 16);  // to the next row block
  const int pitch = a.chunk * kW4K * 2 + 64;  // bytes of a row: rows 2i and 2i + 1 on different banks

  float acc[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][nt][e] = 0.f;

  int row_at[NT];  // a column's activation row (beyond M any: it is not written)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) row_at[nt] = min(nt * 8 + g, a.M - 1) * pitch;
  constexpr int P = R == 1 ? 6 : 4;  // tiles in flight
  uint4 w[P][R];
  uint2 sc[P][R];
  for (int c0 = t0; c0 < t1; c0 += a.chunk) {
    const int c1 = min(c0 + a.chunk, t1), n = c1 - c0;
    const int k0 = c0 + (n * wk >> kw_log), k1 = c0 + (n * (wk + 1) >> kw_log);
    auto fetch = [&](int i, int kt) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (kt < k1 && rb0 + r < a.RB) {  // else nothing that is read, or rows that are not written
          w[i][r] = load_stream(codes + r * codes_step + kt * 32);
          if (fine) sc[i][r] = load_early8(scales + r * scales_step + kt * 32);
          else sc[i][r].x = load_early4(scales + r * scales_step + (kt >> unit_log) * 16);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < P; ++i) fetch(i, k0 + i);
    if (c0 == t0) grid_dependency_wait();  // weights are there since they were loaded; activations may be on their way
    // activations: 16 bytes are 8 k; beyond K zeros (the codes there are 0)
    const int per_row = n * (kW4K / 8), have = min(per_row, a.K / 8 - c0 * (kW4K / 8));
    if (c0 > t0) __syncthreads();  // the last chunk has been read
    for (int m = warp; m < a.M; m += kW4Warps) {
      uint8_t* dst = w4_smem + (size_t)m * pitch;
      const uint16_t* src = a.x + (int64_t)m * a.x_stride + c0 * kW4K;
#pragma unroll 4
      for (int c = lane; c < per_row; c += 32) {
        if (c < have) copy16(dst + c * 16, src + c * 8);
        else *(uint4*)(dst + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (int kt = k0; kt < k1; kt += P) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (kt + i < k1) {
          uint4 b[NT][2];
          const uint8_t* xs = w4_smem + (kt + i - c0) * (kW4K * 2) + 16 * t;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              b[nt][h] = *(const uint4*)(xs + row_at[nt] + 64 * h);
            }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t words[4] = {w[i][r].x, w[i][r].y, w[i][r].z, w[i][r].w};
            float s[2][2];  // [row half][32-k half]
            if (fine) {
              s[0][0] = bf2f(sc[i][r].x & 0xffffu);
              s[0][1] = __uint_as_float(sc[i][r].x & 0xffff0000u);
              s[1][0] = bf2f(sc[i][r].y & 0xffffu);
              s[1][1] = __uint_as_float(sc[i][r].y & 0xffff0000u);
            } else {
              s[0][0] = s[0][1] = bf2f(sc[i][r].x & 0xffffu);
              s[1][0] = s[1][1] = __uint_as_float(sc[i][r].x & 0xffff0000u);
            }
            float c[NT][4];
            auto flush = [&](int h) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][nt][e] = fmaf(c[nt][e], s[e >> 1][h], acc[r][nt][e]);
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t av[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) av[e][j] = widen4(words[2 * h + e] >> (4 * j));
              if (h == 1 && fine) flush(0);  // groups of 32 end inside the tile
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (h == 0 || fine) mma_bf16_first(c[nt], av[0], b[nt][h].x, b[nt][h].y);
                else mma_bf16(c[nt], av[0], b[nt][h].x, b[nt][h].y);
                mma_bf16(c[nt], av[1], b[nt][h].z, b[nt][h].w);
              }
            }
            flush(1);
          }
          fetch(i, kt + i + P);
        }
      }
    }
  }

  float* part = (float*)w4_smem;
  __syncthreads();  // the activations have been read
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(wk * 8 * NT + nt * 8 + 2 * t + (e & 1)) * stride + (wr * R + r) * 16 + g + 8 * (e >> 1)] = acc[r][nt][e];
  __syncthreads();
  const int n0 = cta * cta_rows, shift = 31 - __clz(cta_rows);  // cta_rows is a power of two
  auto put = [&](int m, int n, float v) {
    if (n0 + n < a.N) {
      if (a.y_f32) ((float*)a.y)[(int64_t)m * a.y_stride + n0 + n] = v;
      else ((uint16_t*)a.y)[(int64_t)m * a.y_stride + n0 + n] = f2bf(v);
    }
  };
  // over the k warps, then (all loads at once: each crosses the SMs) over the cluster
  for (int idx = threadIdx.x; idx < cta_rows * a.M; idx += kW4Threads) {
    const int m = idx >> shift, n = idx & (cta_rows - 1);
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kW4Warps; ++k)
      if (k < kw) v += part[(k * 8 * NT + m) * stride + n];
    if (S == 1) put(m, n, v);
    else part[m * stride + n] = v;
  }
  if (S == 1) return;
  cluster.sync();
  for (int idx = rank * kW4Threads + threadIdx.x; idx < cta_rows * a.M; idx += S * kW4Threads) {
    const int m = idx >> shift, n = idx & (cta_rows - 1);
    float v[kW4MaxSplit];
#pragma unroll
    for (int c = 0; c < kW4MaxSplit; ++c) v[c] = c < S ? cluster.map_shared_rank(part, c)[m * stride + n] : 0.f;
#pragma unroll
    for (int c = 1; c < kW4MaxSplit; ++c) v[0] += v[c];
    put(m, n, v[0]);
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

// ---- more rows, on the tcgen05 tensor cores
//
// A CTA takes 128 weight rows (16 a warp) and all activation rows as NCOL columns, a k
// tile of 64 at a time: codes widened to bf16 and activations in shared
// memory with the 128-byte swizzle, a group's partial sums in tensor memory. Two tiles
// later, when their product has run, every warp takes half of its rows' columns, times
// the group's scale, into fp32 registers. CTAs of a cluster split k as above.
//
// Tensor memory: a CTA's four (or fewer) accumulators take 4 NCOL of the 512 columns,
// and shared memory is asked for so that an SM holds two CTAs at most: an allocation
// never waits for a CTA that waits for this one.
//
// 64 x 12288 x 2048 19 us against 29 of the kernel above, 48 x 30000 x 4096 53 against
// 97: bound by the chain of a tile (a product's sums, activations, codes), 0.6 us, which
// two CTAs an SM overlap. A warp of its own issues the products (done by one of the
// widening warps, behind a barrier: 23 and 64 us).
constexpr int kTcThreads = kW4Threads + 32, kTcRows = 128, kTcTries = 1 << 17, NCOL = kW4MaxM;
constexpr int kTcSmem = 80 * 1024;
__global__ void __launch_bounds__(kTcThreads, 2) w4_tc_kernel(const __grid_constant__ W4Args a) {
  extern __shared__ __align__(1024) uint8_t w4_tc_smem[];  // [2] weights, [4] activations; then the sums
  __shared__ uint64_t bars[2], full[2];                    // the products of even, odd tiles have run; their operands are there
  __shared__ uint64_t drained;                             // all products have run
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = 1 << a.s_log, rank = blockIdx.x & (S - 1), cta = blockIdx.x >> a.s_log;
  const int unit_log = a.group == 128 ? 1 : 0;  // k tiles of a group
  const bool fine = a.group == 32;
  const int units = a.KT >> unit_log;
  const int t0 = (units * rank >> a.s_log) << unit_log, n = ((units * (rank + 1) >> a.s_log) << unit_log) - t0;
  uint8_t* const wts = w4_tc_smem;
  uint8_t* const act = w4_tc_smem + 2 * kTcRows * 128;

  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    mbar_init(&full[0], kW4Threads);
    mbar_init(&full[1], kW4Threads);
    mbar_init(&drained, 1);
    mbar_init_fence();
    s_failed = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "n"(4 * NCOL)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // this warp's codes, four tiles ahead; the scales of a thread's row, two tiles ahead of their use
  const bool worker = warp < kW4Warps;  // the last warp issues the products
  const int rb = cta * 8 + warp, row = (warp & 3) * 32 + lane;
  const uint4* codes = a.codes + ((size_t)min(rb, a.RB - 1) * a.KT + t0) * 32 + lane;
  const int rbs = min(cta * 8 + row / 16, a.RB - 1);
  const uint16_t* scales = a.scales + (fine ? ((size_t)rbs * a.sunits + t0) * 32 + scale_slot(row & 15, 0, 32)
                                            : ((size_t)rbs * a.sunits + (t0 >> unit_log)) * 16 + scale_slot(row & 15, 0, 64));
  uint4 w[4];
  uint32_t sc[4] = {0u, 0u, 0u, 0u};
  auto load_scale = [&](uint32_t& v, int i) {
    if (i < n) v = fine ? *(const uint32_t*)(scales + i * 32) : scales[(i >> unit_log) * 16];
  };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n && worker) w[i] = load_stream(codes + i * 32);
  load_scale(sc[0], 0);
  load_scale(sc[1], 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_dependency_wait();  // activations

  // tile i's activations, 16 bytes are 8 k; zeros beyond M and K
  constexpr int kActs = NCOL * 8 / kW4Threads;
  const int act_k = t0 * kW4K + (tid & 7) * 8;
  const uint16_t* act_src[kActs];
  uint32_t act_dst[kActs];
#pragma unroll
  for (int e = 0; e < kActs; ++e) {
    const int m = (e * kW4Threads + tid) >> 3 & (NCOL - 1);
    act_src[e] = m < a.M ? a.x + (int64_t)m * a.x_stride + act_k : nullptr;
    act_dst[e] = smem_addr(act + word_at(m, tid & 7));
  }
  auto load_act = [&](int i) {
    if (i < n) {
      const bool in = act_k + i * kW4K < a.K;
#pragma unroll
      for (int e = 0; e < kActs; ++e)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(act_dst[e] + (i & 3) * (NCOL * 128)),
                     "l"(in && act_src[e] ? act_src[e] + i * kW4K : a.x), "r"(in && act_src[e] ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Bounded; a product that does not end gives NaN. After a failure the loops go on, with
  // waits that give up at once (leaving the loops by a vote cost 3 %).
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return;
#pragma unroll 1
    for (int tries = 0; tries < kTcTries && !*(volatile int*)&s_failed; ++tries)
      if (mbar_test_sleep(bar, parity, 10000)) return;
    *(volatile int*)&s_failed = 1;
  };
  constexpr int kCols = NCOL / 2;  // of a thread
  float acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
  const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * kCols;
  auto accumulator = [&](int i, int half) { return (fine ? 2 * (i & 1) + half : i >> unit_log & 1) * NCOL; };
  auto add = [&](int i, int half, float s) {
#pragma unroll
    for (int c0 = 0; c0 < kCols; c0 += 16) {
      uint32_t v[16];
      tmem_ld16(v, mine + accumulator(i, half) + c0);
      tmem_wait_ld(v);
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[c0 + c] = fmaf(__uint_as_float(v[c]), s, acc[c0 + c]);
    }
  };
  if (!worker) {
    const bool leader = elect_one();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      wait(&full[i & 1], i >> 1 & 1);
      tc_fence_after();
      const uint64_t ad = swizzled_desc(wts + (i & 1) * (kTcRows * 128)), bd = swizzled_desc(act + (i & 3) * (NCOL * 128));
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma(tmem + accumulator(i, ks >> 1), ad + 2 * ks, bd + 2 * ks, tc_idesc_bf16(kTcRows, NCOL),
                 fine ? ks & 1 : ks > 0 || (unit_log && (i & 1)));
        tc_commit(&bars[i & 1]);
      }
      __syncwarp();
    }
    drain_products(&drained, kTcTries);
  } else {
    load_act(0);
    load_act(1);
  }
#pragma unroll 1
  for (int i0 = 0; i0 < n + 2 && worker; i0 += 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u;
      if (i >= n + 2) break;
      if (i >= 2) {  // tile i - 2 has run: its places are free, its sums are there
        wait(&bars[i & 1], ((i >> 1) - 1) & 1);
        tc_fence_after();
        const uint32_t s2 = sc[(u + 2) & 3];
        if (fine) {
          add(i - 2, 0, bf2f(s2 & 0xffffu));
          add(i - 2, 1, __uint_as_float(s2 & 0xffff0000u));
        } else if (!unit_log || (i & 1)) {
          add(i - 2, 0, bf2f(s2));
        }
      }
      load_scale(sc[(u + 2) & 3], i + 2);
      if (i >= n) continue;
      load_act(i + 2);
      const uint32_t words[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      uint8_t* dst = wts + (i & 1) * (kTcRows * 128);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *(uint4*)(dst + word_at(warp * 16 + 8 * r + g, 4 * h + t)) =
              make_uint4(widen4(words[2 * h] >> 4 * r), widen4(words[2 * h] >> (4 * r + 8)), widen4(words[2 * h + 1] >> 4 * r),
                         widen4(words[2 * h + 1] >> (4 * r + 8)));
      if (i + 4 < n) w[u] = load_stream(codes + (i + 4) * 32);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      fence_async_shared();
      tc_fence_before();
      mbar_arrive(&full[i & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(4 * NCOL) : "memory");
  const float poison = s_failed ? __int_as_float(0x7fffffff) : 0.f;
  const int n0 = cta * kTcRows;
  auto put = [&](int m, int r, float v) {
    if (m < a.M && n0 + r < a.N) {
      if (a.y_f32) ((float*)a.y)[(int64_t)m * a.y_stride + n0 + r] = v;
      else ((uint16_t*)a.y)[(int64_t)m * a.y_stride + n0 + r] = f2bf(v);
    }
  };
  float* part = (float*)w4_tc_smem;  // [NCOL][rows + 4]
  constexpr int kPitch = kTcRows + 4;
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    const int m = (warp >> 2) * kCols + c;
    if (!worker) break;
    if (S == 1) put(m, row, acc[c] + poison);
    else part[m * kPitch + row] = acc[c] + poison;
  }
  if (S == 1) return;
  cluster.sync();
#pragma unroll 1
  for (int idx = rank * kTcThreads + tid; idx < kTcRows * a.M; idx += S * kTcThreads) {
    const int m = idx / kTcRows, r = idx % kTcRows;
    float v[kW4MaxSplit];
#pragma unroll
    for (int c = 0; c < kW4MaxSplit; ++c) v[c] = c < S ? cluster.map_shared_rank(part, c)[m * kPitch + r] : 0.f;
#pragma unroll
    for (int c = 1; c < kW4MaxSplit; ++c) v[0] += v[c];
    put(m, r, v[0]);
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

constexpr int kW4Smem = 200 * 1024;  // at most

template <int NT, int R>
cudaError_t w4_setup_one() {
  return cudaFuncSetAttribute(w4_kernel<NT, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4Smem);
}
cudaError_t w4_setup() {
  cudaError_t e;
  (e = w4_setup_one<1, 1>()) || (e = w4_setup_one<2, 1>()) || (e = w4_setup_one<2, 2>()) || (e = w4_setup_one<4, 1>()) ||
      (e = w4_setup_one<8, 2>()) ||
      (e = cudaFuncSetAttribute(w4_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem));
  return e;
}

template <int NT, int R>
cudaError_t w4_launch(W4Args a, cudaStream_t s) {
  const int S = 1 << a.s_log, kw = kW4Warps >> a.rw_log, cta_rows = 16 * R << a.rw_log;
  a.chunk = std::min((a.KT + S - 1) / S, (kW4Smem / a.M - 64) / (kW4K * 2));
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((a.N + cta_rows - 1) / cta_rows * S);
  lc.blockDim = dim3(kW4Threads);
  lc.dynamicSmemBytes = std::max((size_t)a.M * (a.chunk * kW4K * 2 + 64), (size_t)kw * 8 * NT * (cta_rows + 4) * sizeof(float));
  lc.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  lc.numAttrs = 1;
  early_launch(lc, at);
  return cudaLaunchKernelEx(&lc, w4_kernel<NT, R>, a);
}

cudaError_t w4_tc_launch(W4Args a, int sms, cudaStream_t s) {
  const int ctas = (a.RB + 7) / 8;
  a.s_log = 0;
  while ((1 << a.s_log) < kW4MaxSplit && ctas << a.s_log < sms && a.KT >= 8 << a.s_log) ++a.s_log;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(ctas << a.s_log);
  lc.blockDim = dim3(kTcThreads);
  lc.dynamicSmemBytes = kTcSmem;
  lc.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1 << a.s_log;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  lc.numAttrs = 1;
  early_launch(lc, at);
  return cudaLaunchKernelEx(&lc, w4_tc_kernel, a);
}

thread_local ErrorText g_w4_err;  // of calls without a handle

int fail(qtts_w4* w, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  (w ? w->err : g_w4_err).set(fmt, ap);
  va_end(ap);
  return code;
}

// A failed runtime call is reported here, not by a later call's check of the last error.
int cuda_fault(qtts_w4* w, const char* who, cudaError_t e) {
  cudaGetLastError();
  return fail(w, e == cudaErrorMemoryAllocation ? QTTS_E_OOM : QTTS_E_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

struct DeviceBuf {
  void* p = nullptr;
  cudaError_t alloc(size_t n) { return cudaMalloc(&p, n); }
  ~DeviceBuf() {
    if (p && cudaFree(p) != cudaSuccess) cudaGetLastError();
  }
};

}  // namespace
}  // namespace qtts

using namespace qtts;

extern "C" {

const char* qtts_w4_last_error(const qtts_w4* w) { return (w ? w->err : g_w4_err).get(); }

int qtts_w4_create(int N, int K, int group, int device, qtts_w4** out) {
  if (!out) return fail(nullptr, QTTS_E_INVALID, "null argument");
  *out = nullptr;
  if (N < 1 || K < 1) return fail(nullptr, QTTS_E_INVALID, "N and K must be positive");
  if (group != 32 && group != 64 && group != 128) return fail(nullptr, QTTS_E_INVALID, "group must be 32, 64 or 128");
  if (K % group) return fail(nullptr, QTTS_E_INVALID, "K must be a multiple of the group");
  if (N > (1 << 24) || K > (1 << 20)) return fail(nullptr, QTTS_E_INVALID, "N must be at most 2^24 and K at most 2^20");
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) cudaGetLastError();
  if (device < 0 || device >= ndev) return fail(nullptr, QTTS_E_CUDA, "no CUDA device %d", device);
  DeviceGuard g(device);
  if (!g.ok) return fail(nullptr, QTTS_E_CUDA, "cudaSetDevice(%d) failed", device);
  qtts_w4* w = new (std::nothrow) qtts_w4();
  if (!w) return fail(nullptr, QTTS_E_OOM, "out of host memory");
  w->N = N;
  w->K = K;
  w->group = group;
  w->device = device;
  w->RB = (N + kW4Rows - 1) / kW4Rows;
  w->KT = (K + kW4K - 1) / kW4K;
  const size_t ns = (size_t)w->RB * scale_units(w->KT, K, group) * (group == 32 ? 32 : 16);
  cudaError_t e = cudaDeviceGetAttribute(&w->G, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = w4_setup();
  if (e == cudaSuccess) e = cudaMalloc((void**)&w->codes, (size_t)w->RB * w->KT * 512);
  if (e == cudaSuccess) e = cudaMalloc((void**)&w->scales, ns * sizeof(uint16_t));
  if (e == cudaSuccess) e = cudaMemset(w->scales, 0, ns * sizeof(uint16_t));
  if (e != cudaSuccess) {
    qtts_w4_destroy(w);
    return cuda_fault(nullptr, "qtts_w4_create", e);
  }
  *out = w;
  return QTTS_OK;
}

void qtts_w4_destroy(qtts_w4* w) {
  if (!w) return;
  {
    DeviceGuard g(w->device);
    for (void* p : {(void*)w->codes, (void*)w->scales})
      if (p && cudaFree(p) != cudaSuccess) cudaGetLastError();
  }
  delete w;
}

static int w4_fill(qtts_w4* w, const void* src, size_t src_bytes, const void* scales, const char* who) {
  DeviceGuard g(w->device);
  if (!g.ok) return fail(w, QTTS_E_CUDA, "cudaSetDevice failed");
  const size_t nk = (size_t)w->N * w->K, ns = nk / w->group;
  DeviceBuf in, q, s, bad;
  cudaError_t e = in.alloc(src_bytes);
  if (e == cudaSuccess && !scales) e = q.alloc(nk);
  if (e == cudaSuccess) e = s.alloc(ns * sizeof(uint16_t));
  if (e == cudaSuccess) e = bad.alloc(sizeof(int));
  if (e != cudaSuccess) return cuda_fault(w, who, e);
  const int grid = 8 * w->G;
  int flag = 0;
  w->loaded = false;
  // device sources may still be being written on the caller's streams
  e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(in.p, src, src_bytes, cudaMemcpyDefault);
  if (e == cudaSuccess && scales) e = cudaMemcpy(s.p, scales, ns * sizeof(uint16_t), cudaMemcpyDefault);
  if (e == cudaSuccess) e = cudaMemset(bad.p, 0, sizeof(int));
  if (e == cudaSuccess && !scales) {
    w4_quantize_kernel<<<grid, 256>>>((const uint16_t*)in.p, w->N, w->K, w->group, (int8_t*)q.p, (uint16_t*)s.p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    w4_pack_kernel<<<grid, 256>>>((const int8_t*)(scales ? in.p : q.p), (const uint16_t*)s.p, w->N, w->K, w->group,
                                  w->RB, w->KT, w->codes, w->scales, (int*)bad.p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpy(&flag, bad.p, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fault(w, who, e);
  if (flag) return fail(w, QTTS_E_INVALID, "%s: a code outside -8..7", who);
  w->loaded = true;
  return QTTS_OK;
}

int qtts_w4_quantize(qtts_w4* w, const uint16_t* weights) {
  if (!w) return QTTS_E_INVALID;
  if (!weights) return fail(w, QTTS_E_INVALID, "qtts_w4_quantize: null argument");
  return w4_fill(w, weights, (size_t)w->N * w->K * 2, nullptr, "qtts_w4_quantize");
}

int qtts_w4_load(qtts_w4* w, const int8_t* codes, const uint16_t* scales) {
  if (!w) return QTTS_E_INVALID;
  if (!codes || !scales) return fail(w, QTTS_E_INVALID, "qtts_w4_load: null argument");
  return w4_fill(w, codes, (size_t)w->N * w->K, scales, "qtts_w4_load");
}

int qtts_w4_export(qtts_w4* w, int8_t* codes_host, uint16_t* scales_host) {
  if (!w) return QTTS_E_INVALID;
  if (!codes_host || !scales_host) return fail(w, QTTS_E_INVALID, "qtts_w4_export: null argument");
  if (!w->loaded) return fail(w, QTTS_E_STATE, "qtts_w4_export: no weights loaded");
  DeviceGuard g(w->device);
  if (!g.ok) return fail(w, QTTS_E_CUDA, "cudaSetDevice failed");
  const size_t nk = (size_t)w->N * w->K, ns = nk / w->group;
  DeviceBuf q, s;
  cudaError_t e = q.alloc(nk);
  if (e == cudaSuccess) e = s.alloc(ns * sizeof(uint16_t));
  if (e != cudaSuccess) return cuda_fault(w, "qtts_w4_export", e);
  w4_unpack_kernel<<<8 * w->G, 256>>>(w->codes, w->scales, w->N, w->K, w->group, w->KT, (int8_t*)q.p, (uint16_t*)s.p);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpy(codes_host, q.p, nk, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemcpy(scales_host, s.p, ns * sizeof(uint16_t), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fault(w, "qtts_w4_export", e);
  return QTTS_OK;
}

int qtts_w4_linear(qtts_w4* w, int M, const uint16_t* x, int64_t x_stride, void* y, int64_t y_stride, int y_dtype,
                   void* stream) {
  if (!w) return QTTS_E_INVALID;
  if (M < 0 || M > kW4MaxM) return fail(w, QTTS_E_BATCH, "qtts_w4_linear: M = %d outside 0..%d", M, kW4MaxM);
  if (!w->loaded) return fail(w, QTTS_E_STATE, "qtts_w4_linear: no weights loaded");
  if (y_dtype != QTTS_DTYPE_BF16 && y_dtype != QTTS_DTYPE_F32)
    return fail(w, QTTS_E_INVALID, "qtts_w4_linear: y must be bf16 or fp32");
  if (M == 0) return QTTS_OK;
  if (!x || !y) return fail(w, QTTS_E_INVALID, "qtts_w4_linear: null argument");
  if (((uintptr_t)x & 15) || x_stride < w->K || x_stride % 8)
    return fail(w, QTTS_E_INVALID,
                "qtts_w4_linear: x must be 16-byte aligned, with a row stride that is a multiple of 8 and holds a row");
  if (((uintptr_t)y & (y_dtype == QTTS_DTYPE_F32 ? 3 : 1)) || y_stride < w->N)
    return fail(w, QTTS_E_INVALID, "qtts_w4_linear: y must be aligned to its type, with a row stride that holds a row");
  DeviceGuard g(w->device);
  if (!g.ok) return fail(w, QTTS_E_CUDA, "cudaSetDevice failed");
  W4Args a{w->codes, w->scales, w->N, w->K, w->RB, w->KT, w->group, scale_units(w->KT, w->K, w->group),
           M, x, x_stride, y, y_stride, y_dtype == QTTS_DTYPE_F32, 0, 0, 0};
  cudaError_t e;
  const cudaStream_t s = (cudaStream_t)stream;
  // Up to 8 rows: 16 weight rows a CTA, its warps along k (activations are few,
  // weights spread over all SMs), 32 where that fills the SMs four times over
  // (12288 x 2048: 6.7 us against 7.5). More rows: every CTA copies all
  // activations, so as many of its warps along the weight rows as leave about one
  // CTA an SM (24 x 9000 x 4096: 14 us with 4 warps, 18 with 2; 16 x 30000 x 4096
  // 38 with 8, 61 with 2 or 4), and one row block a warp, two where there are few
  // activations and many blocks (12 x 2048 x 6144: 5.9 us with one, 8.1 with two;
  // 16 x 30000 x 4096 80 and 38). Clusters along k until the SMs have a CTA each
  // and while every warp keeps two k tiles. Over 32 rows the tcgen05 kernel where
  // four CTAs for each 128 weight rows are three quarters of the SMs or more (from 3585
  // rows on; 64 x 4096 x 2048: 11.4 us against 15.5; 64 x 2048 x 6144: 26 against 12.7),
  // split as far as K allows: with few k tiles its CTAs are fewer but short (64 x 6144 x
  // 256: 5.4 us against 5.6, 33 rows 5.3 against 4.1; 64 x 12288 x 256 6.1 against 10.8). With 8 to 15 k tiles it
  // is slower than the other kernel where that one's CTAs, one an SM and then not split,
  // are all there at once (64 x 6144 x 512: 9.1 us against 6.6, 33 x 9728 x 768 7.9
  // against 6.3; 64 x 6144 x 1024, two waves: 8.6 against 15.7).
  const int blocks = M <= 8 ? 1 : M <= 16 ? 1 + (w->RB > 2 * w->G) : M <= 32 ? 1 : 2;  // row blocks of a warp
  auto ctas_of = [&](int rw_log) { return (w->RB + (blocks << rw_log) - 1) / (blocks << rw_log); };
  if (M <= 8) {
    a.rw_log = w->RB > 4 * w->G;
  } else {
    a.rw_log = 1;
    const int most = M <= 16 ? w->G * 13 / 10 : M <= 32 ? w->G : 1 << 30;
    while (a.rw_log < 3 && ctas_of(a.rw_log) > most) ++a.rw_log;
  }
  const int kw = kW4Warps >> a.rw_log;
  while ((1 << a.s_log) < kW4MaxSplit && ctas_of(a.rw_log) << a.s_log < w->G && w->KT >= (4 * kw) << a.s_log) ++a.s_log;
  if (M <= 8) e = w4_launch<1, 1>(a, s);
  else if (M <= 16) e = blocks == 1 ? w4_launch<2, 1>(a, s) : w4_launch<2, 2>(a, s);
  else if (M <= 32) e = w4_launch<4, 1>(a, s);
  else if (4 * ((w->RB + 7) / 8 * kW4MaxSplit) >= 3 * w->G && !(w->KT >= 8 && w->KT < 16 && ctas_of(a.rw_log) <= w->G))
    e = w4_tc_launch(a, w->G, s);
  else e = w4_launch<8, 2>(a, s);
  if (e != cudaSuccess) return cuda_fault(w, "qtts_w4_linear", e);
  return QTTS_OK;
}

}  // extern "C"
