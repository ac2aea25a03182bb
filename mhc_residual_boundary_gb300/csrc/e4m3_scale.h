/* e4m3_scale.h -- the scale of an 8-bit block and its inverse from the block's
 * largest magnitude, step for step as elementary FP32 operations give them
 * (plain C, so that the host can run them too):
 *   scale   = amax * (1 / 448)
 *   inverse = (1 / amax) * 448
 * each constant, reciprocal and product rounded to nearest.  PyTorch computes amax
 * / 448 and 448 / amax on a GPU in just these steps, so 8-bit values are the same
 * bits as those of a quantiser written in it.
 *
 * The rounded reciprocal is a Newton step with fused multiply-adds from one within
 * an ulp (P. Markstein, "Computation of elementary functions on the IBM RISC
 * System/6000 processor", IBM J. Res. Dev. 34 (1), 1990).  It rounds to nearest for
 * all divisors but those whose 24 significant bits are all ones, where the
 * neighbour below may come out (1 / amax lies 2^-25 of an ulp above the middle):
 * tests/test_e4m3_scale_host.py tries all significands with every such start.
 */
#ifndef MHC_E4M3_SCALE_H
#define MHC_E4M3_SCALE_H

#ifdef __CUDACC__
#define MHC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#include <math.h>
#define MHC_HOST_DEVICE static inline
#endif

/* amax: from 2^-100 on, infinity and NaN included. */
MHC_HOST_DEVICE float e4m3_scale(float amax) { return amax * (1.f / 448.f); }

/* The divisor is taken 2^20 smaller, so that its reciprocal is a normal number for
 * every finite amax; r0 is that reciprocal within an ulp, of e4m3_divisor(amax).
 * The Newton step is taken at amax itself and rounds once, to a subnormal number
 * where 1 / amax is one. */
MHC_HOST_DEVICE float e4m3_divisor(float amax) { return amax * 0x1p-20f; }
MHC_HOST_DEVICE float e4m3_inverse(float amax, float r0) {
  const float t = r0 * 0x1p-20f, y = fmaf(fmaf(-amax, t, 1.f), t, t);
  /* infinity: 0, NaN: NaN */
  return (amax <= 3.402823466e38f ? y : r0) * 448.f;
}

#endif
