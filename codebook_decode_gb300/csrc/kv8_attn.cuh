// kv8_attn.cuh -- what the two attention kernels over the 8-bit cache share.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kv8.cuh"

namespace qtts {

// How far (in powers of two) a score may pass the running maximum before the
// maximum follows: weights stay below 2^kSlack.
constexpr float kSlack = 6.f;
constexpr float kNone = -1.5e38f;  // running maximum before the first value
constexpr float kLog2e = 1.4426950408889634f;

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
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *(const uint32_t*)&h;
}

// A sum of weights relative to 2^from, relative to 2^to. In two halves: the maxima follow
// weight times V scale, so a first block of zeros (held at 2^-100) leaves a sum of up to
// 2^118 behind, which counts beside large values though the whole factor is below fp32's range.
__device__ __forceinline__ float rebase(float sum, float from, float to) {
  const float half = ex2(0.5f * (from - to));
  return sum * half * half;
}
__device__ __forceinline__ void axpy(float4& v, float4 x, float f) {
  v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
}

}  // namespace qtts
