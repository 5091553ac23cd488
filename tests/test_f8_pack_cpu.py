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
