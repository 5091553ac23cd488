"""Rows to 8 bits, with and without the residual's addition and the root-mean-square norm, against 64 bits."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def rows(R, n, h, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    gain = torch.exp(0.7 * torch.randn(1, h, generator=g))
    return [(std * gain * torch.randn(n, h, generator=g)).to(dt) for _ in range(R)]


SIZES = [(1, 1, 16), (1, 1, 4096), (2, 3, 128), (1, 5, 112), (2, 7, 144), (1, 33, 1008), (4, 9, 2064), (8, 64, 1024), (1, 2, 65536), (1, 200, 5008)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("R,n,h", SIZES)
def test_quantize_is_exact(R, n, h, dt):
    xs = rows(R, n, h, dt, 3 * n + h)
    codes, scales = coc.quantize_f8([x.to(DEV) for x in xs])
    for x, c, s in zip(xs, codes, scales):
        want, e = f8.quantize(x.double())
        assert torch.equal(s.cpu().view(torch.uint8), e.view(torch.uint8))
        assert torch.equal(c.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dt", [BF, HF])
def test_quantize_borders_and_specials(dt):
    x = torch.zeros(12, 256)
    x[0, 0], x[0, 130] = 448.0, 449.0 if dt == HF else 450.0       # on a scale's border, and above it
    x[1] = 2.0 ** -20
    x[2, 5], x[2, 6] = float("inf"), 3.0
    x[3, 5], x[3, 6] = float("-inf"), -3.0
    x[4, 5], x[4, 6] = float("nan"), 3.0
    x[5] = float("nan")
    x[6] = float("inf")
    x[7, :128] = torch.linspace(-448, 448, 128)
    x[8, 0], x[8, 1:128] = 448.0, 2.0 ** -8          # below e4m3's least value beside the largest
    x[9, 0] = torch.finfo(dt).max
    x[10, 0] = torch.finfo(dt).tiny
    x[11, 0] = -torch.finfo(dt).max
    x = x.to(dt)
    codes, scales = coc.quantize_f8([x.to(DEV)])
    f8.check_codes(codes[0], scales[0], x.double(), torch.zeros(12, 256, dtype=torch.float64))
    assert scales[0].cpu().view(torch.uint8)[5, 0] == 27 and scales[0].cpu().view(torch.uint8)[6, 1] == 27   # 2**-100


# fp32: the sum of squares over VPT * 8 values a thread, 5 shuffles and 32 warps, each addition 2**-24, halved by the root;
# rsqrt 2 units, four products: less than 2**-18 in all
NORM_REL = 2.0 ** -18


def check_norm(x, res, w, eps, codes, scale, total, dt):
    s32 = x.float() if res is None else x.float() + res.float()
    if res is not None:
        want = s32.to(dt)
        assert torch.equal(total.cpu().view(torch.int16), want.view(torch.int16))
    s = x.double() if res is None else x.double() + res.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()
    # the sum itself is rounded to 24 bits: 2**-24 of it is within NORM_REL
    f8.check_codes(codes, scale, y, NORM_REL * y.abs())


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("R,n,h", SIZES + [(1, 400, 1024), (1, 170, 8192), (1, 160, 16384), (1, 153, 32784)])
def test_norm(R, n, h, dt, res):
    xs = rows(R, n, h, dt, 5 * n + h)
    rs = rows(R, n, h, dt, 7 * n + h, 2.0) if res else None
    g = torch.Generator().manual_seed(h)
    w = (1.0 + 0.3 * torch.randn(h, generator=g)).to(dt)
    codes, scales, sums = coc.add_rms_norm_f8([x.to(DEV) for x in xs], w.to(DEV), residuals=[r.to(DEV) for r in rs] if res else None, eps=1e-5)
    assert (sums is None) == (not res)
    for r in range(R):
        check_norm(xs[r], rs[r] if res else None, w, float(torch.tensor(1e-5)), codes[r], scales[r], sums[r] if res else None, dt)


@pytest.mark.parametrize("std,eps", [(1e-4, 1e-5), (1e-6, 1e-20), (1e15, 1e-6), (1e25, 1e-6), (3e36, 1e-6), (1.0, 1e10)])
def test_norm_of_small_and_large_values(std, eps):
    h = 640
    xs = rows(1, 9, h, BF, 11, std)
    xs[0][3] = 0.0                                   # a row of zeros among them
    xs[0][4] = rows(1, 1, h, BF, 12)[0][0]           # and an ordinary one
    w = torch.ones(h, dtype=BF)
    codes, scales, _ = coc.add_rms_norm_f8([xs[0].to(DEV)], w.to(DEV), eps=eps)
    check_norm(xs[0], None, w, float(torch.tensor(eps, dtype=torch.float32)), codes[0], scales[0], None, BF)


def test_norm_keeps_bad_rows_to_themselves():
    h = 384
    x = rows(1, 6, h, BF, 2)[0]
    clean, _, _ = coc.add_rms_norm_f8([x.to(DEV)], torch.ones(h, dtype=BF, device=DEV))
    x[1, 7], x[3, 200], x[4, 0] = float("nan"), float("inf"), float("-inf")
    codes, scales, _ = coc.add_rms_norm_f8([x.to(DEV)], torch.ones(h, dtype=BF, device=DEV))
    got = codes[0].cpu().view(torch.uint8)
    for r in (0, 2, 5):
        assert torch.equal(got[r], clean[0].cpu().view(torch.uint8)[r])
    val = f8.real(codes[0], scales[0])
    assert val[1].isnan().all()
    # s / sqrt(inf) is 0 where s is finite and NaN where it is infinite
    for r, at in ((3, 200), (4, 0)):
        assert val[r, at].isnan() and val[r].isnan().sum() == 1 and (val[r].nan_to_num() == 0).all()


def test_norm_in_place_and_given_outputs():
    R, n, h = 2, 5, 272
    xs, rs = [t.to(DEV) for t in rows(R, n, h, BF, 1)], [t.to(DEV) for t in rows(R, n, h, BF, 2)]
    w = torch.ones(h, dtype=BF, device=DEV)
    codes, scales, sums = coc.add_rms_norm_f8(xs, w, residuals=rs)
    keep = [r.clone() for r in rs]
    outs = [torch.empty(n, h, dtype=f8.E4M3, device=DEV) for _ in range(R)]
    ss = [torch.empty(n, 3, dtype=f8.E8M0, device=DEV) for _ in range(R)]
    c2, s2, u2 = coc.add_rms_norm_f8(xs, w, residuals=rs, sums=rs, outs=outs, scales=ss)
    for r in range(R):
        assert u2[r] is rs[r] and c2[r] is outs[r] and not torch.equal(rs[r], keep[r])
        assert torch.equal(rs[r], sums[r])
        assert torch.equal(outs[r].view(torch.uint8), codes[r].view(torch.uint8)) and torch.equal(ss[r].view(torch.uint8), scales[r].view(torch.uint8))
    # the sum over x itself
    c3, s3, u3 = coc.add_rms_norm_f8(xs, w, residuals=keep, sums=xs)
    for r in range(R):
        assert u3[r] is xs[r] and torch.equal(xs[r], sums[r])
        assert torch.equal(c3[r].view(torch.uint8), codes[r].view(torch.uint8)) and torch.equal(s3[r].view(torch.uint8), scales[r].view(torch.uint8))


@pytest.mark.parametrize("R,n,h", [(1, 1, 4096), (8, 3, 144), (2, 700, 4096)])
def test_new_outputs_do_not_overlap(R, n, h):
    """Small new outputs are one allocation, large sums their own: codes, scales and sums of all ranks lie apart."""
    xs, rs = [t.to(DEV) for t in rows(R, n, h, BF, 1)], [t.to(DEV) for t in rows(R, n, h, BF, 2)]
    outs = coc.add_rms_norm_f8(xs, torch.ones(h, dtype=BF, device=DEV), residuals=rs)
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for ts in outs for t in ts)
    assert len(spans) == 3 * R and all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(t.data_ptr() % 16 == 0 for ts in (outs[0], outs[2]) for t in ts)


def test_rows_empty():
    codes, scales = coc.quantize_f8([torch.empty(0, 256, dtype=BF, device=DEV)])
    assert codes[0].shape == (0, 256) and scales[0].shape == (0, 2)
    w = torch.ones(256, dtype=BF, device=DEV)
    codes, scales, sums = coc.add_rms_norm_f8([torch.empty(0, 256, dtype=BF, device=DEV)], w)
    assert codes[0].shape == (0, 256) and sums is None
