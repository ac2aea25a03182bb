"""The scale of an 8-bit block and its inverse (csrc/e4m3_scale.h) against the
host's correctly rounded operations, for every significand, with every reciprocal
within an ulp of the true one to start from.  A significand of all ones, the one
that a Newton step may round to the neighbour below, is counted apart."""
import os
import subprocess

from conftest import ROOT

SOURCE = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include "e4m3_scale.h"
static float of(uint32_t b) { float f; memcpy(&f, &b, 4); return f; }
static uint32_t bits(float f) { uint32_t b; memcpy(&b, &f, 4); return b; }
static long wrong, all_ones;
static void inverse(float amax) {
  volatile float one = 1.f / amax, want = one * 448.f;
  volatile float r = 1.f / e4m3_divisor(amax);
  for (int d = -1; d <= 1; ++d) {
    const float r0 = of(bits(r) + d);
    /* its distance from the true reciprocal, of which an ulp is the gap to the next float */
    const double off = (double)r0 * e4m3_divisor(amax) - 1, ulp = ((double)of(bits(r) + 1) - r) * e4m3_divisor(amax);
    if (off > ulp || off < -ulp) continue;
    const uint32_t got = bits(e4m3_inverse(amax, r0));
    if (got == bits(want)) continue;
    volatile float below = of(bits(one) - 1), low = below * 448.f;
    if ((bits(amax) & 0x7fffffu) == 0x7fffffu && got == bits(low)) ++all_ones;
    else ++wrong;
  }
}
static void scale(float amax) {
  volatile float y = 1.f / 448.f, want = amax * y;
  if (bits(e4m3_scale(amax)) != bits(want)) ++wrong;
}
int main(void) {
  for (uint32_t m = 0; m < 1u << 23; ++m) {
    scale(of(127u << 23 | m));
    inverse(of(127u << 23 | m));
  }
  printf("significands %ld, all ones %d\n", wrong, all_ones <= 2);
  /* every exponent up to 2^126, significands spread over it */
  for (uint32_t e = 27; e < 253; ++e)
    for (uint32_t m = 0; m < 1u << 23; m += 8191) {
      scale(of(e << 23 | m));
      inverse(of(e << 23 | m));
    }
  printf("exponents %ld\n", wrong);
  /* and beyond: every BF16 value */
  for (uint32_t b = 253u << 23; b < 255u << 23; b += 1u << 16) {
    scale(of(b));
    inverse(of(b));
  }
  printf("subnormal reciprocals %ld\n", wrong);
  const float inf = of(0x7f800000u), nan = of(0x7fffffffu);
  printf("infinity %d %d\n", e4m3_scale(inf) == inf, e4m3_inverse(inf, 0.f) == 0.f);
  printf("nan %d %d\n", e4m3_scale(nan) != e4m3_scale(nan), e4m3_inverse(nan, nan) != e4m3_inverse(nan, nan));
  return 0;
}
"""


def test_every_step_is_rounded_to_nearest(tmp_path):
    src, exe = tmp_path / "quotients.c", tmp_path / "quotients"
    src.write_text(SOURCE)
    subprocess.check_call(["gcc", "-std=c11", "-O2", "-ffp-contract=off", "-I",
                           os.path.join(ROOT, "mhc_residual_boundary_gb300", "csrc"), str(src), "-o", str(exe), "-lm"])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out == ["significands 0, all ones 1", "exponents 0", "subnormal reciprocals 0", "infinity 1 1", "nan 1 1"]
