"""Contractions as long as the layers' (k 8192, 8 x 3584) against 64 bits, within what the tensor cores' sums may be off along
their course: 5e-4 of the outputs' size at k 28672 in one range, a tenth of the bound that short products are held to and less.
"""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def make(R, m, n, k, seed, parts=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    gain = torch.exp(0.5 * torch.randn(1, k, generator=g, device=DEV))
    x, xs = zip(*[tuple(t[0] for t in coc.quantize_f8([(torch.randn(m, k, generator=g, device=DEV) * gain).to(BF)])) for _ in range(R)])
    w, ws = zip(*[coc.f8_pack(torch.randn(n, k, generator=g, device=DEV) * k ** -0.5, parts) for _ in range(R)])
    return list(x), list(xs), list(w), list(ws)


@pytest.fixture(params=["0", "1"], ids=["slab", "tile"])
def kernel(request, monkeypatch):
    monkeypatch.setenv("COC_F8_TILE", request.param)
    return request.param


def course(x, xs, w, ws, kernel):
    """Sums and bound; tiles have one range, slabs 1 to 8 (the widest bound of them)."""
    y, off = f8.course(x, xs, w, ws)
    for ranges in range(2, 9) if kernel == "0" else ():
        off = torch.maximum(off, f8.course(x, xs, w, ws, ranges)[1])
    return y, off


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("R,m,n,k", [(8, 1, 264, 3584), (8, 64, 512, 3584), (1, 300, 520, 28672), (2, 130, 264, 4112)])
def test_sums(R, m, n, k, dt, kernel):
    x, xs, w, ws = make(R, m, n, k, m + k)
    out = coc.matmul_all_reduce_f8(x, xs, w, ws, dtype=dt)[0]
    coc.sync_status()
    y, e = course(x, xs, w, ws, kernel)
    unit = 2.0 ** -8 if dt == BF else 2.0 ** -11
    bound = unit * (y.abs() + e) + e + 2.0 ** -25
    err = (out.double() - y).abs()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3f} of the bound"


@pytest.mark.parametrize("m,f,k", [(1, 400, 8192), (64, 272, 8192), (260, 272, 8192)])
def test_gated(m, f, k, kernel):
    x, xs, w, ws = make(1, m, 2 * f, k, m + f, parts=2)
    codes, scales = coc.all_gather_gated_matmul_f8(x, xs, w, ws)
    coc.sync_status()
    fb = f8.blocks(f)
    g, ge = course(x, xs, [w[0][:f]], [ws[0][:fb]], kernel)
    u, ue = course(x, xs, [w[0][f:]], [ws[0][fb:]], kernel)
    silu = g * torch.sigmoid(g)
    # |silu'| <= 1.1; the gate itself 2**-18 as in the short products' test
    off = 1.1 * ge * (u.abs() + ue) + silu.abs() * ue + 2.0 ** -18 * (silu * u).abs() + 2.0 ** -110
    f8.check_codes(codes[0], scales[0], (silu * u).cpu(), off.cpu())
