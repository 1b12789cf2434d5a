"""CPU: the bound on a plan's tiles (csrc/sp_plan.h) that lets a prefill call be
checked before its first launch without making every plan."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_aware_paged_gb300", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("bound")
    src = d / "bound.cpp"
    src.write_text('''#include "sp_plan.h"
using namespace sp;
extern "C" long long bound(long long n) { return plan_tiles_bound(n); }
extern "C" long long tiles(int kind, int sink, int window, int P, const int* idx, int n_idx, long long n_b, long long lo,
                           long long hi) {
    UnitPol u{};
    u.kind = kind; u.sink = sink; u.window = window; u.n_idx = n_idx;
    u.ring = (window + P - 1) / P + 1; u.sink_pages = (sink + P - 1) / P;
    return make_plan(u, idx, n_b, lo, hi, P).ntiles;
}
''')
    so = str(d / "bound.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    ll = ctypes.c_longlong
    lib.bound.restype = lib.tiles.restype = ll
    lib.bound.argtypes = [ll]
    lib.tiles.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ll, ll, ll]
    return lib


def test_no_plan_passes_the_bound(plan):
    rng = np.random.default_rng(1)
    most = 0
    for _ in range(20000):
        P = int(rng.choice([16, 32, 64, 128]))
        n_b = int(rng.choice([0, 1, 127, 128, 129, int(rng.integers(0, 1 << 12)), int(rng.integers(0, 1 << 30))]))
        lo = n_b + 128 * int(rng.integers(0, 4))
        hi = lo + int(rng.integers(0, 128))
        top = int(rng.choice([1, 200, n_b + 600]))
        sink, window = int(rng.integers(0, top)), 1 + int(rng.integers(0, top))
        idx = np.unique(rng.integers(0, hi + 300, 50)).astype(np.int32)
        kind = int(rng.integers(0, 3))
        t = plan.tiles(kind, sink, window, P, idx.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), len(idx), n_b, lo, hi)
        assert t <= plan.bound(hi + 1), (kind, sink, window, P, n_b, lo, hi)
        most = max(most, t)
    assert most > 1 << 22                       # plans that an item cannot count are among them
