"""Sizes whose offsets pass 2**31 elements: the last rows are where they belong."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_rows_past_2_31_values():
    h, n = 65536, 33000                              # 2.16e9 values
    x = torch.zeros(n, h, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(1)
    tail = torch.randn(3, h, generator=g).to(BF)
    x[-3:] = tail.to(DEV)
    codes, scales = coc.quantize_f8([x])
    want, e = f8.quantize(tail.double())
    assert torch.equal(codes[0][-3:].cpu().view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(scales[0][-3:].cpu().view(torch.uint8), e.view(torch.uint8))
    assert (scales[0][:-3].view(torch.uint8) == 27).all()
    w = torch.ones(h, dtype=BF, device=DEV)
    codes, scales, _ = coc.add_rms_norm_f8([x], w, eps=1e-6)
    y = tail.double() / torch.sqrt((tail.double() ** 2).mean(1, keepdim=True) + 1e-6)
    f8.check_codes(codes[0][-3:], scales[0][-3:], y, 2.0 ** -18 * y.abs())


@pytest.mark.parametrize("m,n,k", [(66000, 33000, 32), (140000, 16384, 16)])
def test_products_past_2_31_outputs(m, n, k):
    g = torch.Generator().manual_seed(2)
    x, xs = f8.activation(g, 300, k)
    w, ws = coc.f8_pack(torch.randn(n, k, generator=g))
    codes = torch.zeros(m, k, dtype=torch.uint8, device=DEV)
    scales = torch.full((m, 1), 127, dtype=torch.uint8, device=DEV)
    codes[-300:], scales[-300:] = x.view(torch.uint8).to(DEV), xs.view(torch.uint8).to(DEV)
    out = coc.matmul_all_reduce_f8([codes.view(f8.E4M3)], [scales.view(f8.E8M0)], [w.to(DEV)], [ws.to(DEV)])[0]
    coc.sync_status()
    ref, size = f8.product([x], [xs], [w], [ws])
    e = f8.sum_error(size, k)
    assert ((out[-300:].double().cpu() - ref).abs() <= 2.0 ** -8 * (ref.abs() + e) + e).all()
    assert (out[:64] == 0).all() and (out[-364:-300] == 0).all()
