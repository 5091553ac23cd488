"""The append's lookup of pages (csrc/coc_kv_units.h) compiled for the host:
every page that receives tokens is found once, and nothing else is."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_matmul_collective_gb300", "csrc")
SHIM = """
#include "coc_kv_units.h"
extern "C" int unit_of(const int32_t* cu, const int32_t* lens, int seqs, int tokens, int page, int unit, int* out) {
    coc::AppendUnit u;
    if (!coc::append_unit_of(cu, lens, seqs, tokens, page, unit, u)) return 0;
    out[0] = u.s; out[1] = u.page; out[2] = u.start; out[3] = u.first; out[4] = u.last; out[5] = u.token;
    return 1;
}
"""


@pytest.fixture(scope="module")
def unit_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CSRC}", str(d / "shim.cpp"), "-o", str(d / "units.so")], check=True)
    f = ctypes.CDLL(str(d / "units.so")).unit_of

    def call(cu, lens, tokens, page, unit):
        out = (ctypes.c_int * 6)()
        c = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
        found = f(c, (ctypes.c_int32 * len(lens))(*lens), len(lens), tokens, page, unit, out)
        return tuple(out) if found else None
    return call


def units(cu, seqs, tokens, page):
    return range(seqs if cu is None else tokens // page + 2 * seqs)


def wanted(cu, lens, page):
    """{(sequence, page): (first new position, one past the last, token of position 0)} by the definition."""
    out = {}
    for s, n in enumerate(lens):
        b, e = (s, s + 1) if cu is None else (cu[s], cu[s + 1])
        for t in range(b, e):
            p = n - (e - t)
            if p >= 0:
                lo, hi, at = out.get((s, p // page), (p, p, t - p))
                out[s, p // page] = (min(lo, p), max(hi, p + 1), at)
    return out


def check(unit_of, cu, lens, tokens, page):
    got = {}
    for unit in units(cu, len(lens), tokens, page):
        u = unit_of(cu, lens, tokens, page, unit)
        if u is not None:
            s, j, start, first, last, token = u
            assert start == j * page and start <= first < last <= start + page
            assert (s, j) not in got
            got[s, j] = (first, last, token)
    assert got == wanted(cu, lens, page)


@pytest.mark.parametrize("cu,lens,page", [([64, 65], [1], 16), ([64, 65], [65], 16), ([2048, 2049], [1], 64), ([256, 257], [70], 64),
                                          ([16, 16, 17], [5, 9], 16), ([15, 16, 40], [1, 60], 16), ([1000, 1000], [7], 16)])
def test_offsets_that_do_not_begin_at_zero(unit_of, cu, lens, page):
    """Offsets cut out of a larger batch's."""
    for pad in (0, 1, 100):
        check(unit_of, cu, lens, cu[-1] + pad, page)


@pytest.mark.parametrize("seed", range(60))
def test_batches(unit_of, seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 64, 128])
    seqs = r.randint(1, 9)
    news = [r.choice([0, 0, 1, 1, r.randint(1, 9), r.randint(1, 4 * page)]) for _ in range(seqs)]
    cu = [r.choice([0, 0, r.randint(1, 5 * page)])]
    for n in news:
        cu.append(cu[-1] + n)
    # lengths below the new tokens too: what is ahead of position 0 is not appended
    lens = [max(-1, n + r.choice([0, 0, 1, r.randint(-n, 300)])) for n in news]
    check(unit_of, cu, lens, cu[-1] + r.choice([0, 3, 200]), page)
    check(unit_of, None, lens, seqs, page)


@pytest.mark.parametrize("seed", range(60))
def test_offsets_and_lengths_of_any_kind(unit_of, seed):
    """Descending and out-of-range offsets, lengths up to the largest integer: no table entry and no token outside."""
    r = random.Random(1000 + seed)
    page, seqs, tokens = r.choice([16, 64, 128]), r.randint(1, 6), r.choice([1, 17, 300])
    wild = [-(1 << 31), -1, 0, 1, tokens // 2, tokens, tokens + 1, (1 << 31) - 1]
    cu = [r.choice(wild) for _ in range(seqs + 1)]
    lens = [r.choice([-(1 << 31), -1, 0, 1, page, 5 * page + 1, (1 << 31) - 1, (1 << 31) - page]) for _ in range(seqs)]
    for unit in units(cu, seqs, tokens, page):
        u = unit_of(cu, lens, tokens, page, unit)
        if u is not None:
            s, j, start, first, last, token = u
            assert 0 <= s < seqs and 0 <= j <= (lens[s] - 1) // page
            assert start == j * page and start <= first < last <= min(start + page, lens[s])
            assert 0 <= first + token and last + token <= tokens
