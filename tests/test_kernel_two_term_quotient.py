"""The grouped gradient quantizer forms x/s as fma(x, hi, fl32(x lo)), with hi + lo the
reciprocal of s = fl32(amax/448) from two 128-entry tables scaled by a power of two. The
tables are re-derived here in exact rationals, and a C program with a correctly rounded
fmaf checks that the E4M3 code equals that of the IEEE quotient for every BF16 |x| <= amax
down to 2^-30 of it (smaller quotients round to zero), both signs, at amax exponents over
the range of the path and beyond its upper end; zeros keep their sign."""
import ctypes
import os
import re
import subprocess
from fractions import Fraction

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "fp8_block_scaled_08_b200", "csrc", "fp8q_quant.cu")

C_SRC = r"""
#include <math.h>
static float dec(int c) {
  const int e = (c >> 3) & 15, m = c & 7;
  return e ? ldexpf(1 + m / 8.0f, e - 7) : ldexpf(m / 8.0f, -6);
}
/* nearest code of t by bisection over the 127 finite magnitudes, ties to the even code */
static int enc(float t) {
  const int sign = signbit(t) ? 128 : 0;
  const float a = fabsf(t);
  if (a >= 448.0f) return sign | 0x7e;
  int lo = 0, hi = 0x7e;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (dec(mid) <= a) lo = mid; else hi = mid;
  }
  const float dl = a - dec(lo), dh = dec(hi) - a;
  const int c = dl < dh ? lo : dh < dl ? hi : (lo & 1 ? hi : lo);
  return sign | c;
}
long check(const float *hi, const float *lo, int E, int depth, int drop_lo, long *pairs) {
  long bad = 0;
  for (int i = 0; i < 128; ++i) {
    const float amax = ldexpf(1 + i / 128.0f, E);
    const float s = amax / 448.0f, p = ldexpf(1.0f, -E);
    const float h = hi[i] * p, l = drop_lo ? 0.0f : lo[i] * p;
    for (int d = 0; d <= depth; ++d)
      for (int m = 0; m < 128; ++m)
        for (int sg = 0; sg < 2; ++sg) {
          float x = ldexpf(1 + m / 128.0f, E - d);
          if (x > amax || x < 0x1p-126f) continue;
          if (sg) x = -x;
          const float y = x * l;
          bad += enc(fmaf(x, h, y)) != enc(x / s);
          ++*pairs;
        }
    for (int sg = 0; sg < 2; ++sg) {
      const float x = sg ? -0.0f : 0.0f, y = x * l, t = fmaf(x, h, y);
      bad += t != 0.0f || !signbit(t) != !signbit(x);
    }
  }
  return bad;
}
"""


def table(name):
    txt = open(SRC).read()
    body = re.search(r"__constant__ float %s\[128\] = \{(.*?)\};" % name, txt, re.S).group(1)
    return np.array([float.fromhex(t.strip().rstrip("f")) for t in body.split(",") if t.strip()],
                    np.float32)


def constant(name):
    return int(re.search(r"\b%s = (-?\d+)" % name, open(SRC).read()).group(1))


def test_tables_are_the_reciprocal_in_two_terms():
    hi, lo = table("kRecipHi"), table("kRecipLo")
    assert hi.shape == lo.shape == (128,)
    for i in range(128):
        s = np.float32(np.float32(1 + i / 128.0) / np.float32(448.0))
        exact = 1 / Fraction(float(s))
        assert Fraction(float(hi[i])) <= exact < Fraction(float(np.nextafter(hi[i], np.float32(np.inf))))
        assert lo[i] == np.float32(float(exact - Fraction(float(hi[i])))) and lo[i] >= 0


def test_codes_equal_those_of_the_ieee_quotient(tmp_path):
    src, lib = tmp_path / "two_term.c", tmp_path / "two_term.so"
    src.write_text(C_SRC)
    subprocess.check_call(["gcc", "-O2", "-std=c11", "-fPIC", "-shared", "-ffp-contract=off",
                           "-fno-fast-math", str(src), "-o", str(lib), "-lm"])
    f = ctypes.CDLL(str(lib)).check
    f.restype = ctypes.c_long
    hi, lo = table("kRecipHi"), table("kRecipLo")
    ptr = lambda a: a.ctypes.data_as(ctypes.POINTER(ctypes.c_float))  # noqa: E731
    lo_e, hi_e = constant("kRecipMinExp"), constant("kRecipMaxExp")
    pairs = ctypes.c_long(0)
    for e in (lo_e, lo_e + 1, -40, -1, 0, 1, 30, hi_e - 1, hi_e, hi_e + 8):
        assert f(ptr(hi), ptr(lo), e, 30, 0, ctypes.byref(pairs)) == 0, e
    assert pairs.value > 9_000_000
    # the check can fail: one term alone misses ties
    assert f(ptr(hi), ptr(lo), 0, 30, 1, ctypes.byref(pairs)) > 0
