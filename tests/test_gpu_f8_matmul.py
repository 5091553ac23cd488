"""The fused operators on 8-bit activations and weights, and the gated projections, against float64 products of the same codes."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def weight(g, n, k, parts=1):
    w = torch.randn(n, k, generator=g) * torch.exp(0.5 * torch.randn(n, 1, generator=g)) * k ** -0.5
    return coc.f8_pack(w, parts)


def make(R, m, n, k, seed, parts=1):
    """Rank activations (m rows each) and weights (n rows each), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x, xs = zip(*[f8.activation(g, m, k) for _ in range(R)])
    w, ws = zip(*[weight(g, n, k, parts) for _ in range(R)])
    return list(x), list(xs), list(w), list(ws)


def dev(*lists):
    return [[t.to(DEV) for t in ts] for ts in lists]


def check(out, ref, size, K, dt):
    u = 2.0 ** -8 if dt == BF else 2.0 ** -11
    e = f8.sum_error(size, K)
    bound = u * (ref.abs() + e) + e + (2.0 ** -25 if dt == HF else 0.0)
    err = (out.cpu().double() - ref).abs()
    assert out.shape == ref.shape
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3f} of the bound"


@pytest.fixture(params=["", "0", "1"], ids=["rule", "slab", "tile"])
def kernel(request, monkeypatch):
    """The kernel by its rule, or either one at every size."""
    if request.param:
        monkeypatch.setenv("COC_F8_TILE", request.param)


CASES = [
    # R, m, n, k, dtype: one tile and less, ragged everywhere, many tiles, every number of rows a tile takes
    (1, 1, 8, 16, BF), (1, 1, 128, 128, HF), (1, 3, 136, 144, BF), (2, 2, 264, 512, HF), (1, 16, 1000, 640, BF), (4, 4, 72, 1040, BF),
    (1, 17, 256, 400, HF), (8, 24, 520, 272, BF), (1, 33, 392, 2048, BF), (2, 64, 128, 4112, HF), (1, 65, 640, 256, BF),
    (8, 128, 264, 384, HF), (1, 129, 200, 528, BF), (4, 260, 1032, 256, BF), (1, 300, 24, 16, HF), (2, 514, 384, 1360, BF),
    (1, 1000, 520, 112, BF),
]


@pytest.mark.parametrize("R,m,n,k,dt", CASES)
def test_all_reduce(R, m, n, k, dt, kernel):
    x, xs, w, ws = make(R, m, n, k, m + n + k)
    outs = coc.matmul_all_reduce_f8(*dev(x, xs, w, ws), dtype=dt)
    coc.sync_status()
    ref, size = f8.product(x, xs, w, ws)
    check(outs[0], ref, size, R * k, dt)
    assert len(outs) == R and all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("R,m,n,k,dt", [c for c in CASES if c[1] % c[0] == 0])
def test_reduce_scatter_is_all_reduce_in_rows(R, m, n, k, dt, kernel):
    x, xs, w, ws = make(R, m, n, k, m + n + k)
    d = dev(x, xs, w, ws)
    outs = coc.matmul_reduce_scatter_f8(*d, dtype=dt)
    whole = coc.matmul_all_reduce_f8(*d, dtype=dt)
    coc.sync_status()
    assert all(o.shape == (m // R, n) for o in outs)
    assert torch.equal(torch.cat(outs), whole[0])


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("R,m,n,k,dt", CASES)
def test_all_gather(R, m, n, k, dt, apart, kernel):
    m = -(-m // R)
    x, xs, w, ws = make(R, m, n, k, m + n + k)
    d = dev(x, xs, w, ws)
    if not apart:
        d[0] = list(torch.cat([t.view(torch.uint8) for t in d[0]]).view(R, m, k).view(f8.E4M3).unbind(0))
        d[1] = list(torch.cat([t.view(torch.uint8) for t in d[1]]).view(R, m, -1).view(f8.E8M0).unbind(0))
    outs = coc.all_gather_matmul_f8(*d, dtype=dt)
    coc.sync_status()
    for r in range(R):
        ref, size = f8.product([torch.cat([t.view(torch.uint8) for t in x]).view(f8.E4M3)], [torch.cat([t.view(torch.uint8) for t in xs]).view(f8.E8M0)],
                               w[r:r + 1], ws[r:r + 1])
        check(outs[r], ref, size, k, dt)


GATED = [(1, 1, 16, 16), (1, 1, 1376, 256), (1, 2, 128, 640), (2, 3, 144, 144), (8, 2, 272, 1040), (1, 20, 384, 512), (4, 12, 112, 272), (1, 64, 400, 2064),
         (2, 50, 256, 384), (1, 129, 160, 256), (4, 70, 528, 400), (1, 300, 1280, 128), (2, 257, 640, 1280)]


@pytest.mark.parametrize("R,m,f,k", GATED)
def test_gated(R, m, f, k, kernel):
    x, xs, w, ws = make(R, m, 2 * f, k, m + f + k, parts=2)
    codes, scales = coc.all_gather_gated_matmul_f8(*dev(x, xs, w, ws))
    coc.sync_status()
    xa, sa = torch.cat([t.view(torch.uint8) for t in x]).view(f8.E4M3), torch.cat([t.view(torch.uint8) for t in xs]).view(f8.E8M0)
    fb = f8.blocks(f)
    for r in range(R):
        g, gsize = f8.product([xa], [sa], [w[r][:f]], [ws[r][:fb]])
        u, usize = f8.product([xa], [sa], [w[r][f:]], [ws[r][fb:]])
        silu = g * torch.sigmoid(g)
        # |silu'| <= 1.1; e^-g, the sum, the quotient and the product: 2**-18 of h for |g| up to 30 (the argument of
        # the exponential is rounded to 2**-24 of itself)
        off = 1.1 * f8.sum_error(gsize, k) * (u.abs() + f8.sum_error(usize, k)) + silu.abs() * f8.sum_error(usize, k) + 2.0 ** -18 * (silu * u).abs() + 2.0 ** -120
        f8.check_codes(codes[r], scales[r], silu * u, off, f"rank {r}")


def test_scales_of_every_kind_reach_their_values(kernel):
    """Codes of one value, scales that differ by row, block and position in the word: exact sums of powers of two."""
    m, n, k = 40, 256, 128 * 11
    g = torch.Generator().manual_seed(5)
    x = torch.ones(m, k).to(f8.E4M3)
    w = torch.ones(n, k).to(f8.E4M3)
    xe = torch.randint(120, 134, (m, 11), generator=g, dtype=torch.uint8)
    we = torch.randint(120, 134, (2, 11), generator=g, dtype=torch.uint8)
    outs = coc.matmul_all_reduce_f8(*dev([x], [xe.view(f8.E8M0)], [w], [we.view(f8.E8M0)]), dtype=BF)
    ref, size = f8.product([x], [xe.view(f8.E8M0)], [w], [we.view(f8.E8M0)])
    check(outs[0], ref, size, k, BF)


@pytest.mark.parametrize("a,b", [(0, 0), (27, 27), (1, 254), (254, 1), (100, 200), (247, 27)])
def test_extreme_scales(a, b, kernel):
    """The product of the scales is taken in the range of fp32: it overflows or goes to nothing only where the result does."""
    m, n, k = 3, 16, 256
    g = torch.Generator().manual_seed(a + b)
    x, _ = f8.activation(g, m, k)
    w, _ = weight(g, n, k)
    xs, ws = torch.full((m, 2), a, dtype=torch.uint8).view(f8.E8M0), torch.full((1, 2), b, dtype=torch.uint8).view(f8.E8M0)
    out = coc.matmul_all_reduce_f8(*dev([x], [xs], [w], [ws]), dtype=BF)[0]
    ref, size = f8.product([x], [xs], [w], [ws])
    check(out, ref, size, k, BF)


def test_nan_and_bad_scales_stay_in_their_rows(kernel):
    m, n, k = 20, 264, 384
    x, xs, w, ws = make(1, m, n, k, 9)
    clean = coc.matmul_all_reduce_f8(*dev(x, xs, w, ws))[0].cpu()
    x[0].view(torch.uint8)[3, 200] = 0x7F             # a NaN code
    xs[0].view(torch.uint8)[7, 1] = 255               # a NaN scale
    ws[0].view(torch.uint8)[1, 2] = 255               # and one of 128 weight rows
    out = coc.matmul_all_reduce_f8(*dev(x, xs, w, ws))[0].cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[3] = bad[7] = True
    bad[:, 128:256] = True
    assert out[bad].isnan().all()
    assert torch.equal(out[~bad], clean[~bad])


def test_inner_zero_writes_zeros(kernel):
    x, w = torch.empty(5, 0, dtype=f8.E4M3, device=DEV), torch.empty(24, 0, dtype=f8.E4M3, device=DEV)
    xs, ws = torch.empty(5, 0, dtype=f8.E8M0, device=DEV), torch.empty(1, 0, dtype=f8.E8M0, device=DEV)
    out = [torch.full((5, 24), 7.0, dtype=BF, device=DEV)]
    coc.matmul_all_reduce_f8([x], [xs], [w], [ws], outs=out)
    assert (out[0] == 0).all()
    # more tiles than the GPU takes at once
    x, w = torch.empty(2300, 0, dtype=f8.E4M3, device=DEV), torch.empty(16384, 0, dtype=f8.E4M3, device=DEV)
    xs, ws = torch.empty(2300, 0, dtype=f8.E8M0, device=DEV), torch.empty(128, 0, dtype=f8.E8M0, device=DEV)
    out = [torch.full((2300, 16384), 7.0, dtype=BF, device=DEV)]
    coc.matmul_all_reduce_f8([x], [xs], [w], [ws], outs=out)
    codes, scales = coc.all_gather_gated_matmul_f8([x], [xs], [w], [ws.view(torch.uint8).new_empty(128, 0).view(f8.E8M0)])
    coc.sync_status()
    assert (out[0] == 0).all() and (codes[0].view(torch.uint8) == 0).all() and (scales[0].view(torch.uint8) == 27).all()


def test_runs_give_the_same_bits(kernel):
    x, xs, w, ws = make(2, 40, 520, 4112, 3)
    d = dev(x, xs, w, ws)
    first = coc.matmul_all_reduce_f8(*d)[0].clone()
    for _ in range(5):
        assert torch.equal(coc.matmul_all_reduce_f8(*d)[1], first)
