"""The keys' rotation ``x c + y s`` to the last bit of fp32, on the host: the function's own lines out of ``q2_cache.cu``,
with a number type whose ``*`` is fused into every ``+`` and ``-`` behind it, as the device's compiler may do with plain
operators (and never does with explicitly rounded ones), against exact rational numbers."""
import ctypes
import os
import re
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_q2_gb300", "csrc", "q2_cache.cu")
HOST = """
#include <cmath>
struct Num {
  float v, a, b;
  bool product;
  Num(float x = 0.f) : v(x), a(0.f), b(0.f), product(false) {}
  operator float() const { return v; }
};
static Num operator-(const Num& x) { Num r(-x.v); r.a = -x.a; r.b = x.b; r.product = x.product; return r; }
static Num operator*(const Num& x, const Num& y) { Num r(x.v * y.v); r.a = x.v; r.b = y.v; r.product = true; return r; }
static Num operator+(const Num& x, const Num& y) {
  return x.product ? std::fmaf(x.a, x.b, y.v) : y.product ? std::fmaf(y.a, y.b, x.v) : x.v + y.v;
}
static Num operator-(const Num& x, const Num& y) { return x + -y; }
static Num fma_rn(const Num& x, const Num& y, const Num& z) { return std::fmaf(x.v, y.v, z.v); }
static Num __fmul_rn(const Num& x, const Num& y) { return x.v * y.v; }
static Num __fadd_rn(const Num& x, const Num& y) { return x.v + y.v; }
static Num __fsub_rn(const Num& x, const Num& y) { return x.v - y.v; }
#define __device__
#define __forceinline__ static
#define fmaf fma_rn
#define __fmaf_rn fma_rn
#define float Num
%s
#undef float
extern "C" void turn(int n, const float* x, const float* c, const float* y, const float* s, float* r) {
  for (int i = 0; i < n; ++i) r[i] = turn_exact(x[i], c[i], y[i], s[i]).v;
}
"""


@pytest.fixture(scope="module")
def turn(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    body = re.search(r"__device__ __forceinline__ float turn_exact\(.*?\n}\n", open(SOURCE).read(), re.S).group(0)
    at = tmp_path_factory.mktemp("turn")
    (at / "turn.cpp").write_text(HOST % body)
    subprocess.run(["g++", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-o", str(at / "turn.so"), str(at / "turn.cpp")], check=True)
    return ctypes.CDLL(str(at / "turn.so")).turn


def test_every_bit(turn):
    rng = np.random.default_rng(0)
    n = 20000
    a = rng.uniform(0, 2 * np.pi, n)
    c, s = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    x, y = (rng.normal(size=n).astype(np.float16).astype(np.float32) for _ in range(2))
    x[::2] = np.clip(-y * s / c, -9, 9).astype(np.float16)[::2]                 # half of them nearly cancel
    r = np.empty_like(x)
    p = lambda t: t.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    turn(n, p(x), p(c), p(y), p(s), p(r))
    wrong = 0
    for i in range(n):
        want = Fraction(float(x[i])) * Fraction(float(c[i])) + Fraction(float(y[i])) * Fraction(float(s[i]))
        off = abs(Fraction(float(r[i])) - want)
        near = min(abs(Fraction(float(np.nextafter(r[i], np.float32(t)))) - want) for t in (-np.inf, np.inf))
        wrong += off > near                                                     # a neighbour is nearer
    assert wrong == 0, f"{wrong} of {n}"
