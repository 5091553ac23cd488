"""The 8-bit products' plan (csrc/coc_f8_plan.h) compiled for the host."""
import ctypes
import os
import subprocess

import pytest

import __graft_entry__ as entry

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_matmul_collective_gb300", "csrc")
SHIM = """
#include "coc_f8_plan.h"
static coc::KnownCount known[9];
extern "C" void forget() { for (auto& k : known) k.~KnownCount(), new (&k) coc::KnownCount(); }
// room[k]: what the device says of clusters of k; asked[k] counts the questions; room[k] < 0: an error
extern "C" int ranges(long long tiles, int total, int sms, const int* room, int* asked, int* out) {
    return coc::f8_ranges(tiles, total, sms, [&](int k, int* n) -> int {
        if (known[k].get(n)) return 0;
        ++asked[k];
        if (room[k] < 0) return -room[k];
        known[k].set(*n = room[k]);
        return 0;
    }, out);
}
extern "C" int tiles(int gathers, int gated, int R, long long m, long long n, long long k) { return coc::f8_tiles_sooner(gathers, gated, R, m, n, k, 152); }
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text("#include <new>\n" + SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CSRC}", str(d / "shim.cpp"), "-o", str(d / "plan.so")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


def ranges(shim, tiles, total, room, asked=None):
    asked = asked if asked is not None else (ctypes.c_int * 9)()
    out = ctypes.c_int(0)
    st = shim.ranges(ctypes.c_longlong(tiles), total, 152, (ctypes.c_int * 9)(*room), asked, ctypes.byref(out))
    return st, out.value


ROOM = [0, 152, 76, 50, 36, 28, 24, 18, 16]


def test_ranges_fill_the_gpu(shim):
    shim.forget()
    assert ranges(shim, 1, 32, ROOM) == (0, 8)
    assert ranges(shim, 1, 3, ROOM) == (0, 3)           # no more than there are runs
    assert ranges(shim, 1, 1, ROOM) == (0, 1)
    assert ranges(shim, 32, 32, ROOM) == (0, 4)
    assert ranges(shim, 64, 56, ROOM) == (0, 2)
    assert ranges(shim, 77, 56, ROOM) == (0, 1)
    assert ranges(shim, 37, 56, ROOM) == (0, 3)         # 4 x 37 = 148 SMs, but 36 clusters of 4


def test_a_cluster_that_never_fits_is_asked_for_once_and_never_taken(shim):
    """The same ranges in the first call and in every later one."""
    shim.forget()
    asked = (ctypes.c_int * 9)()
    room = [0, 152, 0, 0, 0, 0, 0, 0, 0]
    for _ in range(3):
        assert ranges(shim, 1, 32, room, asked) == (0, 1)
    assert list(asked)[2:] == [1] * 7


def test_an_error_is_handed_on_and_not_remembered(shim):
    shim.forget()
    asked = (ctypes.c_int * 9)()
    assert ranges(shim, 1, 2, [0, 152, -7] + [0] * 6, asked)[0] == 7
    assert ranges(shim, 1, 2, ROOM, asked) == (0, 2) and asked[2] == 2


def test_smoke_runs_both_kernels(shim):
    """The products of smoke()'s feed-forward block: slabs at its first number of rows, tiles of CTA pairs at its second, by the rule."""
    R, hidden, f = entry.SMOKE_MLP["R"], entry.SMOKE_MLP["hidden"], entry.SMOKE_MLP["ffn"] // entry.SMOKE_MLP["R"]
    for rows, want in zip(entry.SMOKE_MLP["rows"], (0, 1)):
        m = ctypes.c_longlong(R * rows)
        assert shim.tiles(1, 1, R, m, ctypes.c_longlong(f), ctypes.c_longlong(hidden)) == want
        assert shim.tiles(0, 0, R, m, ctypes.c_longlong(hidden), ctypes.c_longlong(f)) == want
