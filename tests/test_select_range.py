"""The arithmetic by which the block selection finds its least selected key (csrc/select_range.cuh),
compiled for the host: the search as the kernel runs it, against a sort."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_gqa_decode_kv_gb300", "csrc")

SOURCE = r"""
#include "select_range.cuh"
// The kernel's loop over one slice.  got: lo, hi, the keys of [lo, hi] still wanted, whether all of
// them are, passes.  Returns 0, or 1 where a pass found no bin.
extern "C" int search(const uint32_t *keys, int n, int need, uint32_t *got) {
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int i = 0; i < n; ++i) {
    if (keys[i] < lo) lo = keys[i];
    if (keys[i] > hi) hi = keys[i];
  }
  bool all = false;
  int pass = 0;
  for (; pass < pgd::kRangePasses && !all && lo != hi; ++pass) {
    int hist[pgd::kRangeBins] = {};
    const int shift = pgd::range_shift(lo, hi);
    for (int i = 0; i < n; ++i)
      if (keys[i] >= lo && keys[i] <= hi) {
        const uint32_t bin = (keys[i] - lo) >> shift;
        if (bin >= (uint32_t)pgd::kRangeBins) return 2;
        ++hist[bin];
      }
    int over = 0, bin = pgd::kRangeBins - 1;
    for (; bin >= 0 && over + hist[bin] < need; --bin) over += hist[bin];
    if (bin < 0) return 1;
    need -= over;
    all = hist[bin] == need;
    pgd::narrow_range(lo, hi, (uint32_t)bin, shift);
  }
  got[0] = lo, got[1] = hi, got[2] = (uint32_t)need, got[3] = all, got[4] = (uint32_t)pass;
  return 0;
}
extern "C" void keys(uint32_t *bits, int n) {
  for (int i = 0; i < n; ++i) bits[i] = pgd::score_key(bits[i]);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("select_range")
    (at / "search.cpp").write_text(SOURCE)
    so = str(at / "search.so")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-I" + CSRC,
                    str(at / "search.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.search.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    lib.keys.argtypes = [ctypes.c_void_p, ctypes.c_int]
    return lib


def _check(lib, keys, need):
    keys = np.ascontiguousarray(keys, dtype=np.uint32)
    got = np.zeros(5, dtype=np.uint32)
    assert lib.search(keys.ctypes.data, len(keys), need, got.ctypes.data) == 0
    lo, hi, left, all_, passes = (int(x) for x in got)
    ordered = np.sort(keys.astype(np.int64))[::-1]
    k = keys.astype(np.int64)
    assert lo <= hi and passes <= 4
    above, inside = int((k > hi).sum()), int(((k >= lo) & (k <= hi)).sum())
    assert lo <= ordered[need - 1] <= hi
    assert above + left == need and 1 <= left <= inside
    assert lo == hi or (all_ and left == inside)


def _order(f):
    """A float's bits as an unsigned integer of the same order."""
    u = np.asarray(f, dtype=np.float32).view(np.uint32)
    return np.where(u >> 31, ~u, u | np.uint32(0x80000000))


@pytest.mark.parametrize("share", [0.0, 0.02, 0.4, 0.98])
@pytest.mark.parametrize("top", [np.inf, np.nan, 3.4e38, 1.8e38, 1e30, 1.0])
def test_search_with_keys_at_the_top_of_the_range(lib, top, share):
    """Ordinary scores of both signs, a share of them `top`: the ends of a bin then lie beyond
    2^32."""
    r = np.random.default_rng(int(share * 100) + 1)
    for _ in range(100):
        f = r.standard_normal(100).astype(np.float32) * np.float32(2.0 ** r.integers(-90, 90))
        f[r.random(100) < share] = top
        if share:
            f[r.integers(100)] = top
        _check(lib, _order(f), int(r.integers(1, 100)))


def test_search_over_every_kind_of_key(lib):
    r = np.random.default_rng(5)
    for n in (1, 2, 3, 17, 256, 3000):
        for _ in range(60):
            span = 2 ** int(r.integers(1, 33))
            first = int(r.integers(0, 2 ** 32 - span + 1))
            keys = (first + r.integers(0, span, n)).astype(np.uint32)
            if r.random() < 0.5:
                keys = keys[r.integers(0, n, n)]
            _check(lib, keys, int(r.integers(1, n + 1)))
    ends = np.array([0, 1, 0x7FFFFFFF, 0x80000000, 0xFEFFFFFF, 0xFF000000, 0xFF000001, 0xFFFFFFFE,
                     0xFFFFFFFF], dtype=np.uint32)
    for _ in range(500):
        keys = ends[r.integers(0, len(ends), 12)]
        _check(lib, keys, int(r.integers(1, 13)))


def test_keys_keep_the_order_of_scores(lib):
    r = np.random.default_rng(9)
    f = np.concatenate([r.standard_normal(4000) * 2.0 ** r.integers(-140, 127, 4000),
                        [0.0, np.inf, -np.inf, 3.4e38, -3.4e38, 1e-45, -1e-45]]).astype(np.float32)
    k = f.copy().view(np.uint32)
    lib.keys(k.ctypes.data, len(k))
    o = np.argsort(f, kind="stable")
    assert (np.diff(k[o].astype(np.int64))[np.diff(f[o]) > 0] > 0).all()
    assert (k > 0).all()
