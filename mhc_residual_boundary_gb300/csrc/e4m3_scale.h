/* e4m3_scale.h -- the two quotients of an 8-bit block, amax / 448 and 448 /
 * amax, correctly rounded to FP32 with a handful of fused multiply-adds (plain C,
 * so that the host can run them too).
 *
 * Markstein's correction (P. Markstein, "Computation of elementary functions on
 * the IBM RISC System/6000 processor", IBM J. Res. Dev. 34 (1), 1990): with y =
 * 1 / b rounded to nearest and q within an ulp of a / b, r = a - b q is exact in
 * one fused multiply-add and q + r y rounds to a / b rounded.  A reciprocal
 * within an ulp is brought to the nearest one by a Newton step; no divisor is left
 * out, as all 2^23 significands were tried with all such reciprocals
 * (tests/test_e4m3_scale_host.py).
 */
#ifndef MHC_E4M3_SCALE_H
#define MHC_E4M3_SCALE_H

#ifdef __CUDACC__
#define MHC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#include <math.h>
#define MHC_HOST_DEVICE static inline
#endif

/* amax / 448 for an amax from 2^-100 on, infinity and NaN included (for these
 * r is not a number). */
MHC_HOST_DEVICE float e4m3_scale(float amax) {
  const float y = 1.f / 448.f;
  const float q = amax * y, r = fmaf(-448.f, q, amax);
  return amax <= 3.402823466e38f ? fmaf(r, y, q) : q;
}

/* 448 / amax.  The divisor is taken 2^20 smaller, so that its reciprocal is a
 * normal number for every finite amax from 2^-100 on; r0 is that reciprocal
 * within an ulp, of e4m3_divisor(amax). */
MHC_HOST_DEVICE float e4m3_divisor(float amax) { return amax * 0x1p-20f; }
MHC_HOST_DEVICE float e4m3_inverse(float amax, float r0) {
  const float b = e4m3_divisor(amax), a = 448.f * 0x1p-20f;
  const float y = fmaf(fmaf(-b, r0, 1.f), r0, r0);
  const float q = a * y;
  /* infinity: 0, NaN: NaN */
  return amax <= 3.402823466e38f ? fmaf(fmaf(-b, q, a), y, q) : 448.f * r0;
}

#endif
