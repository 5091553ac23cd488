"""Packing of a model's own weights."""
import torch

from tensor_matmul_collective_gb300 import coc


def test_pack_of_a_parameter_keeps_no_graph():
    w = torch.nn.Parameter(torch.randn(200, 272, generator=torch.Generator().manual_seed(1)))
    codes, scales = coc.f8_pack(w)
    assert not codes.requires_grad and codes.grad_fn is None and not scales.requires_grad
    plain, plain_scales = coc.f8_pack(w.detach())
    assert torch.equal(codes.view(torch.uint8), plain.view(torch.uint8)) and torch.equal(scales.view(torch.uint8), plain_scales.view(torch.uint8))
    assert w.requires_grad and w.grad is None


def test_pack_of_an_empty_inner_size():
    """What the products take at k = 0, and no rows."""
    for n, k, parts in ((24, 0, 1), (2 * 144, 0, 2), (0, 256, 1), (0, 0, 1)):
        codes, scales = coc.f8_pack(torch.zeros(n, k), parts)
        assert codes.shape == (n, k) and codes.dtype == torch.float8_e4m3fn
        assert scales.shape == (parts * -(-n // parts // 128), -(-k // 128)) and scales.dtype == torch.float8_e8m0fnu
