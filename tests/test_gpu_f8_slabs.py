"""The slab kernel where tiles outnumber SMs (two blocks on an SM, a ring of half its shared memory), and where it asks L2 for
weights ahead of the wait for the kernel before (40 MiB of weights and one row tile), which may be writing them."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from test_gpu_f8_long import make
from test_gpu_f8_tiles import check, joined
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def slabs(monkeypatch):
    monkeypatch.setenv("COC_F8_TILE", "0")


# 161 tiles and more; k whole blocks (3-D boxes) and not; from 40 MiB on with weights ahead of the wait
@pytest.mark.parametrize("R,m,n,k,dt", [(1, 5, 20488, 1040, BF), (1, 24, 20488, 2048, HF), (1, 50, 20488, 2064, BF), (1, 64, 20488, 2048, BF),
                                        (1, 100, 20488, 1040, HF), (1, 128, 20488, 2064, BF), (2, 200, 10248, 1280, BF), (4, 60, 19464, 528, BF)])
def test_more_tiles_than_sms(R, m, n, k, dt):
    x, xs, w, ws = make(R, m, n, k, m + n)
    outs = coc.matmul_all_reduce_f8(x, xs, w, ws, dtype=dt)
    coc.sync_status()
    check(outs[0], *f8.product_on(x, xs, w, ws), R * k, dt)
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("R,m,f,k", [(1, 5, 20496, 528), (1, 24, 20496, 1040), (1, 60, 20496, 1040), (8, 8, 2576, 1280), (2, 50, 10256, 528)])
def test_more_gated_tiles_than_sms(R, m, f, k):
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


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("own", [True, False])
def test_weights_that_the_kernel_before_writes(own, gated):
    """The weights' codes are rewritten on the same stream directly ahead of the product, by a kernel that lets the product begin
    under its end (own) or by a copy: the product reads the new ones, every time."""
    n, k, m = 20480, 2560, 40
    g = torch.Generator(device=DEV).manual_seed(3)
    values = [(torch.randn(n, k, generator=g, device=DEV) * s).to(BF) for s in (0.05, 0.04, 0.03)]
    made = [coc.quantize_f8([v])[0][0].clone() for v in values]
    ws = torch.full((n // 128, k // 128), 120, dtype=torch.uint8, device=DEV).view(f8.E8M0)
    x, xs = coc.quantize_f8([torch.randn(m, k, generator=g, device=DEV).to(BF)])
    w = torch.zeros(n, k, dtype=torch.uint8, device=DEV).view(f8.E4M3)
    row_scales = torch.zeros(n, k // 128, dtype=torch.uint8, device=DEV).view(f8.E8M0)

    def product():
        if gated:
            codes, scales = coc.all_gather_gated_matmul_f8(x, xs, [w], [ws])
            return torch.cat([codes[0].view(torch.uint8), scales[0].view(torch.uint8)], 1)
        return coc.matmul_all_reduce_f8(x, xs, [w], [ws])[0]

    def write(i):
        if own:
            coc.quantize_f8([values[i]], outs=[w], scales=[row_scales])
        else:
            w.view(torch.uint8).copy_(made[i].view(torch.uint8))
    want = []
    for i in range(3):
        write(i)
        torch.cuda.synchronize()
        want.append(product())
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = []
    for j in range(30):
        write(j % 3)
        got.append(product())
    coc.sync_status()
    assert all(torch.equal(t, want[j % 3]) for j, t in enumerate(got))
