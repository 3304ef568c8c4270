"""The search for the border between kept and dropped keys, compiled for the host from the
header that the eviction kernels use, over lists of every shape: the border must lie inside
the list's bounds, split it as wanted, and be exact only where it does."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "border_search.cuh"
extern "C" uint32_t find(const uint32_t *keys, int n, uint32_t lo, uint32_t hi, uint32_t want, int *exact) {
    bool e;
    const uint32_t b = nvfp4kv::search_listed(lo, hi, want, e, [&](uint32_t border, int bit, int, uint32_t (&c)[4]) {
        for (uint32_t x = 1; x < 4; x++) {
            c[x] = 0;
            for (int i = 0; i < n; i++) c[x] += keys[i] >= (border | (x << bit));
        }
    });
    *exact = e;
    return b;
}
"""


@pytest.fixture(scope="module")
def find(tmp_path_factory):
    d = tmp_path_factory.mktemp("border")
    (d / "f.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                    "-I", os.path.join(ROOT, "nvfp4_quantised_paged_gb300", "csrc"), str(d / "f.cpp"), "-o", str(d / "f.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "f.so"))
    lib.find.restype = ctypes.c_uint32
    lib.find.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p]

    def call(keys, lo, hi, want):
        k, e = np.ascontiguousarray(keys, np.uint32), ctypes.c_int()
        return lib.find(k.ctypes.data, k.size, lo, hi, want, ctypes.byref(e)), bool(e.value)
    return call


def _check(find, keys, lo, hi, want):
    border, exact = find(keys, lo, hi, want)
    assert lo <= border < hi, (lo, border, hi)   # below lo lie keys that no one counted
    at_least, above = int((keys >= border).sum()), int((keys > border).sum())
    if exact:
        assert at_least == want
    else:                                        # a listed key: of the rows that have it the first ones are taken
        assert (keys == border).any() and above < want <= at_least


@pytest.mark.parametrize("span", [1, 2, 3, 4, 5, 64, 1000, 4096, 1 << 20, 1 << 31])
def test_border_stays_inside_the_list(find, span):
    rng = np.random.default_rng(span)
    for trial in range(60):
        lo = int(rng.integers(1, (1 << 32) - span))
        if trial % 3 == 0:
            lo = max(4096, lo & ~4095) if lo + span < (1 << 32) - 4096 else lo   # borders as a sample gives them
        hi = lo + span
        n = int(rng.integers(1, 200))
        keys = rng.integers(lo, hi, n, dtype=np.uint64).astype(np.uint32)
        for want in {1, n, max(1, n - 1), (n + 1) // 2}:
            _check(find, keys, lo, hi, want)


def test_the_whole_list_is_wanted(find):
    """The first trials lie below lo here: each counts the whole list."""
    for lo, hi in ((0xBF801000, 0xBF9FFFFF), (0x80000FFF, 0xC0000000), (0x7FFFFFFF, 0x80000001), (5, 0xFFFFFFFF)):
        keys = np.array([lo, lo + 1, hi - 1, lo + (hi - lo) // 2], np.uint32)
        border, exact = find(keys, lo, hi, 4)
        assert lo <= border and (exact or border == lo)
        _check(find, np.unique(keys), lo, hi, len(np.unique(keys)))
