"""The tile kernel where a pair of CTAs takes several tiles (over 2 x 76 of them, on 152 SMs): both accumulators, the columns they
share, rings and scale words that go on from tile to tile; and row tiles in more than one group, the odd ones' columns backwards."""
import pytest
import torch

import f8_util as f8
from test_gpu_f8_long import make
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def check(out, y, size, K, dt, what=""):
    e = f8.sum_error(size, K)
    bound = (2.0 ** -8 if dt == BF else 2.0 ** -11) * (y.abs() + e) + e + 2.0 ** -25
    err = (out.double() - y).abs()
    assert out.shape == y.shape and (err <= bound).all(), f"{what} worst {float((err / bound).max()):.3f} of the bound"


# rows, columns, k of a rank; 187 to 198 tiles of 3 to 11 k-blocks a rank in one group of rows, then 18 row tiles in groups of 8, 8 and 2
# (groups are of 1024 / k-blocks of all ranks, at least 8)
SUMMED = [(1, 2600, 4104, 1296, BF), (4, 2600, 4104, 336, HF), (8, 4600, 2056, 2048, BF)]


@pytest.mark.parametrize("R,m,n,k,dt", SUMMED)
def test_summed_products(monkeypatch, R, m, n, k, dt):
    monkeypatch.setenv("COC_F8_TILE", "1")
    x, xs, w, ws = make(R, m, n, k, m + n)
    outs = coc.matmul_all_reduce_f8(x, xs, w, ws, dtype=dt)
    parts = coc.matmul_reduce_scatter_f8(x, xs, w, ws, dtype=dt)
    coc.sync_status()
    assert all(torch.equal(o, outs[0]) for o in outs) and torch.equal(torch.cat(parts), outs[0])
    check(outs[0], *f8.product_on(x, xs, w, ws), R * k, dt)
    for _ in range(3):
        assert torch.equal(coc.matmul_all_reduce_f8(x, xs, w, ws, dtype=dt)[R - 1], outs[0])


def joined(ts, dt):
    return torch.cat([t.view(torch.uint8) for t in ts]).view(dt)


@pytest.mark.parametrize("R,m,n,k,dt", [(2, 1300, 2056, 1296, HF), (2, 2300, 1032, 16384, BF)])
def test_gathered_products(monkeypatch, R, m, n, k, dt):
    monkeypatch.setenv("COC_F8_TILE", "1")
    x, xs, w, ws = make(R, m, n, k, m + n)
    outs = coc.all_gather_matmul_f8(x, xs, w, ws, dtype=dt)
    coc.sync_status()
    for r in range(R):
        check(outs[r], *f8.product_on([joined(x, f8.E4M3)], [joined(xs, f8.E8M0)], w[r:r + 1], ws[r:r + 1]), k, dt, f"rank {r}")


@pytest.mark.parametrize("R,m,f,k", [(1, 2600, 2064, 1296), (2, 1300, 1040, 656), (2, 2300, 528, 16384)])
def test_gated_products(monkeypatch, R, m, f, k):
    monkeypatch.setenv("COC_F8_TILE", "1")
    x, xs, w, ws = make(R, m, 2 * f, k, m + f, parts=2)
    codes, scales = coc.all_gather_gated_matmul_f8(x, xs, w, ws)
    coc.sync_status()
    fb, xa, sa = f8.blocks(f), joined(x, f8.E4M3), joined(xs, f8.E8M0)
    for r in range(R):
        g, gsize = f8.product_on([xa], [sa], [w[r][:f]], [ws[r][:fb]])
        u, usize = f8.product_on([xa], [sa], [w[r][f:]], [ws[r][fb:]])
        silu, ge, ue = g * torch.sigmoid(g), f8.sum_error(gsize, k), f8.sum_error(usize, k)
        off = 1.1 * ge * (u.abs() + ue) + silu.abs() * ue + 2.0 ** -18 * (silu * u).abs() + 2.0 ** -110       # as in test_gpu_f8_matmul.py
        f8.check_codes(codes[r], scales[r], (silu * u).cpu(), off.cpu(), f"rank {r}")
    again, again_scales = coc.all_gather_gated_matmul_f8(x, xs, w, ws)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again + again_scales, codes + scales))
