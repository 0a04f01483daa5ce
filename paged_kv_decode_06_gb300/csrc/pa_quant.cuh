// Arithmetic shared by the cache-write kernels: IEEE quotients by a scale that
// stays fixed over many values, fp8 conversion, bf16 magnitude maxima.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "pa_pack.cuh"

namespace pa {

__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Division by a scale that stays fixed over many values: the IEEE
// round-to-nearest quotient x / s formed from the correctly rounded reciprocal
// r = 1/s by Markstein's correction step (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990; also Muller et al., "Handbook of Floating-Point
// Arithmetic", division with a fused multiply-add): q0 = x r rounded, the
// remainder x - q0 s exact by one FMA, and q0 + (x - q0 s) r rounded once.
// Kept from q0: a zero quotient (its sign: the correction's sum of zeros
// would be +0) and |q0| >= 1024 or NaN (the e4m3 code saturates at 448 either
// way, and an infinite q0 would make the remainder NaN).  Outside
// 2^-64 <= |s| <= 2^64 the plain IEEE division is used.  Checked equal to
// __fdiv_rn (quotients on [2^-20, 1000] and e4m3 codes everywhere) over every
// fp32 x, for every scale amax / 448 of a positive finite bf16 amax and 10000
// random scales (and, for a set of scales, by tests/test_cache_write_div_gpu.py).
struct ScaleDiv {
  float s, r;
  bool fast;
};

__device__ __forceinline__ ScaleDiv scale_div(float s) {
  ScaleDiv d;
  d.s = s;
  d.r = __frcp_rn(s);
  d.fast = fabsf(s) >= 5.421010862427522e-20f && fabsf(s) <= 1.8446744073709552e+19f;   // 2^-64 .. 2^64
  return d;
}

// (a, b) / s on the fast path, two at a time (packed f32x2 arithmetic, each
// half rounded as its scalar form would be).
__device__ __forceinline__ void div_by2(const ScaleDiv& d, float a, float b, float& qa, float& qb) {
  const uint64_t x = f2_pack(a, b);
  const uint64_t r2 = f2_pack(d.r, d.r), ns2 = f2_pack(-d.s, -d.s);
  const uint64_t q0 = fmul2(x, r2);
  const uint64_t q1 = ffma2(ffma2(q0, ns2, x), r2, q0);
  float a0, b0, a1, b1;
  f2_unpack(q0, a0, b0);
  f2_unpack(q1, a1, b1);
  qa = (a0 == 0.f || !(fabsf(a0) < 1024.f)) ? a0 : a1;
  qb = (b0 == 0.f || !(fabsf(b0) < 1024.f)) ? b0 : b1;
}

// Integer quotient of an index by a per-call divisor: 32-bit when the index
// range fits (every practical call), 64-bit otherwise (a uniform branch).
__device__ __forceinline__ int64_t cw_div(int64_t a, int64_t b, bool narrow) {
  return narrow ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Largest of two pairs of 16-bit unsigned integers, half by half.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace pa
