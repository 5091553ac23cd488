"""Sizes at which a 32-bit offset would wrap."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_w4_word_rows_of_4_gib():
    """n = 2**28: a step's four word rows are 2**32 bytes.  Every row holds one code, its own."""
    n, ks = 1 << 28, 64
    w = torch.tensor([0x11111111 * (i + 1) if i < 7 else -0x77777778 for i in range(8)], dtype=torch.int32, device=DEV)
    w = w[:, None].expand(8, n).contiguous()
    x = torch.zeros(1, ks, dtype=torch.bfloat16, device=DEV)
    x[0, 0::8] = torch.tensor([1.0, 2, 4, 8, 16, 32, 64, 128], device=DEV).to(torch.bfloat16)
    out = coc.matmul_all_reduce_w4a16([x], [w], [torch.ones(1, n, dtype=torch.bfloat16, device=DEV)], 64)[0]
    coc.sync_status()
    want = sum(2.0 ** i * (i + 1 - 8) for i in range(8))
    assert torch.tensor(want).to(torch.bfloat16).item() == want
    assert out.min().item() == want and out.max().item() == want
