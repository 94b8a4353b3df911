"""The key interval of the histogram selects (csrc/rkv_bins.h), compiled for the host: the
rounds end, and end on the interval that holds the boundary (no GPU)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from two_stage_kv_snapkv_gb300 import build_lib

# The selects' loop over the same two functions; -1: it did not end within the rounds that
# 32-bit keys and ten bits a round can take.
SOURCE = r"""
#include <string.h>
#include "rkv_bins.h"
extern "C" int rounds(const uint32_t* keys, int n, int k, int cand, uint32_t* lo_, uint32_t* hi_, int* need_, int* nin_) {
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = 0; i < n; ++i) {
    if (keys[i] < lo) lo = keys[i];
    if (keys[i] > hi) hi = keys[i];
  }
  int need = k, nin = n, r = 0;
  while (nin > cand && lo != hi) {
    if (++r > 5) return -1;
    const int shift = rkv::tk_shift(hi - lo);
    if (((hi - lo) >> shift) >= (uint32_t)rkv::kTkBins) return -2;
    uint32_t hist[rkv::kTkBins];
    memset(hist, 0, sizeof hist);
    for (int i = 0; i < n; ++i)
      if (keys[i] >= lo && keys[i] <= hi) ++hist[(keys[i] - lo) >> shift];
    int above = 0, b = rkv::kTkBins - 1;
    while (b > 0 && above + (int)hist[b] < need) above += hist[b--];
    const uint32_t nlo = lo + ((uint32_t)b << shift);
    hi = rkv::tk_upper(nlo, hi, shift);
    lo = nlo;
    need -= above;
    nin = hist[b];
  }
  *lo_ = lo, *hi_ = hi, *need_ = need, *nin_ = nin;
  return r;
}
"""


@pytest.fixture(scope="module")
def rounds(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("bins")
    src, lib = d / "bins.cpp", d / "bins.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + os.path.join(build_lib.CSRC), str(src), "-o",
                    str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).rounds
    u32p, i32p = ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_int32)
    fn.argtypes = [u32p, ctypes.c_int, ctypes.c_int, ctypes.c_int, u32p, u32p, i32p, i32p]
    return fn


def _float_key(x):
    u = ctypes.c_uint32.from_buffer(ctypes.c_float(x)).value
    return ~u & 0xffffffff if u >> 31 else u | 0x80000000


def _check(rounds, keys, k, cand):
    n = len(keys)
    lo, hi, need, nin = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_int32(), ctypes.c_int32()
    r = rounds((ctypes.c_uint32 * n)(*keys), n, k, cand, lo, hi, need, nin)
    assert r >= 0, f"n={n} k={k}: the rounds do not end"
    lo, hi, need, nin = lo.value, hi.value, need.value, nin.value
    edge = sorted(keys, reverse=True)[k - 1]
    assert lo <= edge <= hi, "the boundary key lies outside the interval"
    assert nin == sum(lo <= u <= hi for u in keys) and (nin <= cand or lo == hi)
    assert need == k - sum(u > hi for u in keys) and 1 <= need <= nin


@pytest.mark.parametrize("cand", [32, 64])
def test_more_keys_at_the_top_of_the_range_than_are_taken(rounds, cand):
    rng = random.Random(3)
    for _ in range(400):
        n = rng.randint(cand + 2, 900)
        top = rng.randint(cand + 1, n)
        k = rng.randint(1, min(top, n - 1))
        keys = [0xffffffff] * top + [_float_key(rng.uniform(1e-6, 4.0)) for _ in range(n - top)]
        rng.shuffle(keys)
        _check(rounds, keys, k, cand)


@pytest.mark.parametrize("cand", [32, 64])
def test_any_keys(rounds, cand):
    rng = random.Random(4)
    kinds = [lambda: rng.getrandbits(32), lambda: _float_key(rng.gauss(0, 1)), lambda: _float_key(rng.expovariate(1)),
             lambda: rng.choice([0, 0xffffffff, 0x80000000, 0x7fffffff]), lambda: 0xffffffff - rng.randint(0, 3000),
             lambda: rng.randint(0, 3000), lambda: 0xffffffff - (rng.getrandbits(22) << 10 & 0xffffffff)]
    for i in range(700):
        n = rng.randint(2, 700)
        keys = [kinds[i % len(kinds)]() for _ in range(n)]
        _check(rounds, keys, rng.randint(1, n - 1), cand)
