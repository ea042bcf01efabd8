"""The fixed-point weights of pi_token_sample (csrc/serve/sample_weight.cuh), compiled
for the host: their error against long double.

A weight is 2^-t = 2^(-b/32) (1 - q 2^-36), q a whole number, the sum of two rounded to
the nearest: 1/2 each.  The rest is what fp32 leaves of 1 - e^-z in z < 0.0217, computed
as a sum of two numbers whose low one is below 2^-16, with some eight roundings on the
way: 8 x 2^-16 x 2^-24 x 2^36 = 1/32, and the part of t that has one rounding of
2^-18 x 2^-24 four times over.  A quarter covers it: |error of q| < 1.25, so that a weight
is exact to 1.25 / 2^36 / 2^(-1/32) < 2^-35 of itself.
"""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "activation_sparse_decode_rank_gb300", "csrc", "serve", "sample_weight.cuh")

HARNESS = r"""
#include "%s"
#include <cstdint>
static uint64_t s;
static double rnd() { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return (s >> 11) * 0x1p-53; }
static long double exact_q(float top, float x, float T, int b) {
  const long double r = ((long double)top - x) * 1.442695040888963407359924681001892137L / T - b / 32.L;
  return -expm1l(-r * 0.693147180559945309417232121458176568L) * 0x1p36L;
}
// Largest error of q, in units, of n random logits whose t is in [t0, 64); the largest
// is at (out[0..2]) = (top, x, T).  T's and the maximum's exponents are spread over
// [T0, T1] and up to T 2^spread.
extern "C" double worst(uint64_t seed, long n, double t0, double T0, double T1, double spread, double* out) {
  s = seed * 0x9E3779B97F4A7C15ull + 1;
  double most = 0;
  for (long i = 0; i < n; ++i) {
    const float T = (float)exp2(T0 + (T1 - T0) * rnd());
    const float top = (float)((rnd() < 0.5 ? -1. : 1.) * T * exp2(spread * rnd()));
    const float x = (float)(top - (t0 + (64 - t0) * rnd()) * T / 1.4426950408889634);
    pis::Weights w;
    w.set(top, T, -INFINITY);
    const int b = w.bin(x);
    if (b == pis::kBins) continue;
    const long double e = fabsl((long double)w.q(x, b) - exact_q(top, x, T, b));
    if (!((double)e <= most)) {
      most = (double)e;
      out[0] = top, out[1] = x, out[2] = T;
    }
  }
  return most;
}
extern "C" int one(float top, float x, float T, int* q) {
  pis::Weights w;
  w.set(top, T, -INFINITY);
  const int b = w.bin(x);
  *q = b == pis::kBins ? 0 : w.q(x, b);
  return b;
}
extern "C" double error(float top, float x, float T) {
  int q;
  const int b = one(top, x, T, &q);
  return (double)(q - exact_q(top, x, T, b));
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("weights")
    (d / "w.cpp").write_text(HARNESS % HEADER)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-x", "c++",
                    "-o", str(d / "w.so"), str(d / "w.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "w.so"))
    lib.worst.restype = lib.error.restype = ctypes.c_double
    lib.worst.argtypes = [ctypes.c_uint64, ctypes.c_long] + [ctypes.c_double] * 4 + [ctypes.POINTER(ctypes.c_double)]
    lib.one.argtypes = [ctypes.c_float] * 3 + [ctypes.POINTER(ctypes.c_int)]
    lib.error.argtypes = [ctypes.c_float] * 3
    return lib


@pytest.mark.parametrize("t0,T0,T1,spread", [(0, -2, 2.3, 4), (32, -2, 2.3, 8), (60, -2, 2.3, 8), (32, -60, 60, 30),
                                             (48, 0, 1, 0)])
def test_weight_error(host, t0, T0, T1, spread):
    at = (ctypes.c_double * 3)()
    e = host.worst(7, 400000, t0, T0, T1, spread, at)
    assert 0 < e < 1.25, (e, list(at))


@pytest.mark.parametrize("top,x,T", [(4.79208, -61.81355, 1.50659), (2.55906963, -24.059103, 0.607149661),
                                     (-86.2891769, -218.576263, 3.03540301)])
def test_weights_with_a_long_low_part(host, top, x, T):
    # t near 64, its low part near its largest: the square of z's low part counts
    assert abs(host.error(top, x, T)) < 1.25


@pytest.mark.parametrize("T0,T1", [(60, 68), (68, 121), (110, 121)])
def test_weight_error_at_large_temperatures(host, T0, T1):
    # log2(e) / T keeps its two parts; 44 T, the largest difference that counts, stays finite
    at = (ctypes.c_double * 3)()
    e = host.worst(8, 400000, 32, T0, T1, 0, at)
    assert 0 < e < 1.25, (e, list(at))


def test_differences_past_the_largest_float(host):
    q = ctypes.c_int()
    for T, t in ((1e38, 8.6561702), (3e38, 2.8853901), (3.4e38, 2.5459324)):
        assert host.one(3e38, -3e38, T, ctypes.byref(q)) == int(32 * t)
        assert abs(host.error(3e38, -3e38, T)) < 1.25
    assert host.one(3e38, -3e38, 2.0 ** 64, ctypes.byref(q)) == 2048  # weighs nothing
    assert host.one(3e38, -3e38, 1e19, ctypes.byref(q)) == 2048


def test_largest_weight(host):
    q = ctypes.c_int()
    for top in (0.0, -3.5, 1e30, -1e-30):
        assert host.one(top, top, 0.7, ctypes.byref(q)) == 0 and q.value == 0
