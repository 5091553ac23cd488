"""The gate where e^-g leaves fp32's range: silu(g) is far from nothing beside a large up projection."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

GATES = [0.0, 1.0, -1.0, 30.0, 88.0, 160.0, -30.0, -60.0, -68.0, -69.0, -70.0, -72.0, -80.0, -88.0, -96.0, -104.0, -120.0, -144.0, -160.0, -208.0, -448.0]


@pytest.mark.parametrize("exp", [0, 30, 60, 100, 118])
@pytest.mark.parametrize("tile", ["0", "1"])
def test_gate_over_the_whole_range(monkeypatch, tile, exp):
    """Every column one gate value (a sum of two e4m3 values), every block of 128 one of them, so that its codes show it; sums are exact."""
    monkeypatch.setenv("COC_F8_TILE", tile)
    k, f, rows = 128, 128 * len(GATES), 5
    x = torch.zeros(rows, k)
    x[:, 0] = x[:, 1] = x[:, 2] = 1.0
    w = torch.zeros(2 * f, k)
    for i, g in enumerate(GATES):
        hi = float(torch.tensor(g).to(f8.E4M3).float())
        w[128 * i:128 * i + 128, 0], w[128 * i:128 * i + 128, 1] = hi, g - hi
    w[f:, 2] = torch.tensor([1.0, 1.25, -1.5, 1.75]).repeat(f // 4)
    one = torch.full((rows, 1), 127, dtype=torch.uint8).view(f8.E8M0)
    scales = torch.full((2 * len(GATES), 1), 127, dtype=torch.uint8)
    scales[len(GATES):] = 127 + exp
    codes = x.to(f8.E4M3), w.to(f8.E4M3)
    assert torch.equal(codes[1].float(), w)
    got, got_scales = coc.all_gather_gated_matmul_f8([codes[0].to(DEV)], [one.to(DEV)], [codes[1].to(DEV)], [scales.view(f8.E8M0).to(DEV)])
    coc.sync_status()
    g = (w[:f, 0] + w[:f, 1]).double()
    h = (g / (1.0 + torch.exp(-g)) * w[f:, 2].double() * 2.0 ** exp).expand(rows, f)
    # the argument of 2^x has a relative 2**-24 of up to 231 from the constant log2(e) and as much from its rounding, ln 2 of that in
    # the result; 2^x, the reciprocal and the products 2**-20 more: less than 2**-15 in all.  From g = -170 on nothing is
    # left of 2^-246 and 2^7 for g: with u < 2^121, less than half of the least code, 2**-110
    f8.check_codes(got[0], got_scales[0], h, 2.0 ** -15 * h.abs() + (h.abs() < 2.0 ** -110) * 2.0 ** -110)


@pytest.mark.parametrize("tile", ["0", "1"])
def test_far_gates_leave_the_others_their_bits(monkeypatch, tile):
    """One row whose gates are far out among ordinary rows, which share its warps."""
    monkeypatch.setenv("COC_F8_TILE", tile)
    g = torch.Generator().manual_seed(2)
    k, f, rows = 256, 272, 70
    w = torch.randn(2 * f, k, generator=g)
    w[:f, 0], w[f:, 0] = -8.0, 1.0
    x = torch.randn(rows, k, generator=g)
    x[:, 0] = 0.0
    wc, ws = coc.f8_pack(w, 2)
    got = []
    for first in (0.0, 32.0):                       # row 40: gates near -256
        x[40, 0] = first
        c, s = f8.quantize(x.double())
        codes, scales = coc.all_gather_gated_matmul_f8([c.to(DEV)], [s.to(DEV)], [wc.to(DEV)], [ws.to(DEV)])
        got.append(torch.cat([codes[0].cpu().view(torch.uint8), scales[0].cpu().view(torch.uint8)], 1))
    coc.sync_status()
    other = torch.arange(rows) != 40
    assert torch.equal(got[0][other], got[1][other]) and not torch.equal(got[0][40], got[1][40])
