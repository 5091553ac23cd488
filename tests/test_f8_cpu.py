"""Refusals of the 8-bit calls, which come before any CUDA call, and the packing of weights."""
import ctypes

import pytest
import torch

import f8_util as f8
from tensor_matmul_collective_gb300 import coc

A = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    from tensor_matmul_collective_gb300 import build
    build.build()
    return coc.lib()


def ptrs(*vals):
    return (ctypes.c_void_p * len(vals))(*vals)


def test_quantize_refusals(L):
    p = ptrs(A, A)

    def call(R=2, rows=4, h=256, x=p, codes=p, scale=p, dt=1):
        return L.coc_quantize_f8(R, rows, h, x, codes, scale, dt, None)
    assert call(R=3) == call(R=0) == call(R=16) == coc.ERR_INVALID_ARG
    assert call(dt=2) == coc.ERR_INVALID_ARG
    assert call(h=136) == coc.ERR_ALIGN
    assert call(rows=-1) == call(h=-16) == call(rows=1 << 31) == coc.ERR_SHAPE
    assert call(rows=1 << 30, h=1024) == coc.ERR_SHAPE           # 2^33 scales
    assert call(x=ptrs(A, None)) == call(codes=None) == call(scale=None) == call(scale=ptrs(None, A)) == coc.ERR_INVALID_ARG
    assert call(x=ptrs(A, A + 8)) == call(codes=ptrs(A + 4, A)) == coc.ERR_ALIGN
    assert call(rows=0) == call(h=0) == coc.OK


def test_norm_refusals(L):
    p = ptrs(A, A)

    def call(R=2, rows=4, h=256, x=p, res=p, w=A, eps=1e-6, total=p, codes=p, scale=p, dt=1):
        return L.coc_add_rms_norm_f8(R, rows, h, x, res, w, eps, total, codes, scale, dt, None)
    assert call(R=5) == call(dt=-1) == coc.ERR_INVALID_ARG
    assert call(h=65536 + 16) == coc.ERR_SHAPE
    assert call(h=24) == coc.ERR_ALIGN
    for eps in (0.0, -1.0, 1e-30, float("nan"), float("inf")):
        assert call(eps=eps) == coc.ERR_INVALID_ARG
    assert call(res=None) == call(total=None) == coc.ERR_INVALID_ARG     # one without the other
    assert call(w=None) == coc.ERR_INVALID_ARG
    assert call(w=A + 2) == call(res=ptrs(A, A + 2)) == call(total=ptrs(A + 8, A)) == coc.ERR_ALIGN
    assert call(rows=0, res=None, total=None) == coc.OK


@pytest.mark.parametrize("gated", [False, True])
def test_matmul_refusals(L, gated):
    p = ptrs(A, A)

    def call(op=0, R=2, m=4, n=256, k=256, x=p, xs=p, w=p, ws=p, out=p, scale=p, dt=1):
        if gated:
            return L.coc_all_gather_gated_matmul_f8(R, m, n, k, x, xs, w, ws, out, scale, None)
        return L.coc_fused_matmul_f8(op, R, m, n, k, x, xs, w, ws, out, dt, None)
    assert call(R=3) == coc.ERR_INVALID_ARG
    assert call(k=264) == coc.ERR_ALIGN
    assert call(n=1004) == coc.ERR_ALIGN
    assert call(m=-1) == call(n=1 << 31) == call(k=1 << 31) == coc.ERR_SHAPE
    assert call(m=(1 << 31) - 1024, n=1 << 20) == coc.ERR_SHAPE
    for kw in ({"x": ptrs(A, None)}, {"w": None}, {"xs": None}, {"ws": ptrs(A, None)}, {"out": ptrs(None, A)}):
        assert call(**kw) == coc.ERR_INVALID_ARG, kw
    for kw in ({"x": ptrs(A, A + 8)}, {"w": ptrs(A + 1, A)}, {"out": ptrs(A, A + 8)}):
        assert call(**kw) == coc.ERR_ALIGN, kw
    assert call(m=0) == call(n=0) == coc.OK
    if gated:
        assert call(n=24) == coc.ERR_ALIGN
        assert call(scale=None) == call(scale=ptrs(A, None)) == coc.ERR_INVALID_ARG
        assert call(n=1 << 30) == coc.ERR_SHAPE                  # 2^31 weight rows
    else:
        assert call(dt=2) == call(op=3) == call(op=4) == call(op=-1) == coc.ERR_INVALID_ARG
        assert call(op=1, m=5) == coc.ERR_SHAPE


def test_binding_refuses_cpu_tensors():
    x = [torch.zeros(2, 256, dtype=torch.bfloat16)]
    with pytest.raises(ValueError):
        coc.quantize_f8(x)
    with pytest.raises(ValueError):
        coc.add_rms_norm_f8(x, x[0][0])
    with pytest.raises(ValueError):
        coc.quantize_f8([])
    c, s = coc.f8_pack(torch.zeros(256, 256))
    for call in (coc.matmul_all_reduce_f8, coc.matmul_reduce_scatter_f8, coc.all_gather_matmul_f8, coc.all_gather_gated_matmul_f8):
        with pytest.raises(ValueError):
            call([c[:4]], [s[:1]], [c], [s])


@pytest.mark.parametrize("n,k,parts", [(128, 128, 1), (1, 16, 1), (300, 272, 1), (200, 400, 2), (2 * 1376, 144, 2), (256, 256, 2)])
def test_pack(n, k, parts):
    g = torch.Generator().manual_seed(n + k)
    w = torch.randn(n, k, generator=g) * torch.exp(torch.randn(n, 1, generator=g))
    w[0, 0] = 448.0                                   # on a border
    codes, scales = coc.f8_pack(w, parts)
    half = n // parts
    assert codes.shape == (n, k) and scales.shape == (parts * f8.blocks(half), f8.blocks(k))
    for p in range(parts):
        for b in range(f8.blocks(half)):
            for c in range(f8.blocks(k)):
                t = w[p * half + b * 128:p * half + min(half, b * 128 + 128), c * 128:c * 128 + 128].double()
                e = f8.scale_exp(t.abs().max())
                assert int(scales.view(torch.uint8)[p * f8.blocks(half) + b, c]) == int(e) + 127
                got = codes[p * half + b * 128:p * half + min(half, b * 128 + 128), c * 128:c * 128 + 128].double()
                assert torch.equal(got, f8.round_e4m3(t / f8.pow2(e)))


def test_pack_of_zeros_and_bad_values():
    w = torch.zeros(130, 144)
    w[0, 0], w[129, 0], w[0, 130] = float("inf"), float("nan"), -float("inf")
    codes, scales = coc.f8_pack(w)
    assert (scales.view(torch.uint8) == 27).all()
    c = codes.float()
    assert c[0, 0] == 448 and c[0, 130] == -448 and c[129, 0].isnan() and c.nan_to_num().abs().sum() == 896
    with pytest.raises(ValueError):
        coc.f8_pack(w[:129], 2)
