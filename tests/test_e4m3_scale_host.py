"""The quotients of an 8-bit block (csrc/e4m3_scale.h) against the correctly
rounded divisions of the host, for every significand, with every reciprocal that
the hardware's instruction may give (within an ulp)."""
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
static long wrong;
static void inverse(float amax) {
  volatile float want = 448.f / amax;
  volatile float r = 1.f / e4m3_divisor(amax);
  for (int d = -1; d <= 1; ++d)
    if (bits(e4m3_inverse(amax, of(bits(r) + d))) != bits(want)) ++wrong;
}
static void scale(float amax) {
  volatile float want = amax / 448.f;
  if (bits(e4m3_scale(amax)) != bits(want)) ++wrong;
}
int main(void) {
  for (uint32_t m = 0; m < 1u << 23; ++m) {
    scale(of(127u << 23 | m));
    inverse(of(127u << 23 | m));
  }
  printf("significands %ld\n", wrong);
  /* the ends of the range: every exponent, significands spread over it */
  for (uint32_t e = 27; e < 255; ++e)
    for (uint32_t m = 0; m < 1u << 23; m += 8191) {
      scale(of(e << 23 | m));
      inverse(of(e << 23 | m));
    }
  scale(of(0x7f7fffffu));
  inverse(of(0x7f7fffffu));
  printf("exponents %ld\n", wrong);
  const float inf = of(0x7f800000u), nan = of(0x7fffffffu);
  printf("infinity %d %d\n", e4m3_scale(inf) == inf, e4m3_inverse(inf, 0.f) == 0.f);
  printf("nan %d %d\n", e4m3_scale(nan) != e4m3_scale(nan), e4m3_inverse(nan, nan) != e4m3_inverse(nan, nan));
  return 0;
}
"""


def test_quotients_are_correctly_rounded(tmp_path):
    src, exe = tmp_path / "quotients.c", tmp_path / "quotients"
    src.write_text(SOURCE)
    subprocess.check_call(["gcc", "-std=c11", "-O2", "-ffp-contract=off", "-I",
                           os.path.join(ROOT, "mhc_residual_boundary_gb300", "csrc"), str(src), "-o", str(exe), "-lm"])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out == ["significands 0", "exponents 0", "infinity 1 1", "nan 1 1"]
