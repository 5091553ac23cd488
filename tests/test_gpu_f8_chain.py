"""w8A16 products in a row with 8-bit and 16-bit ones, without waits: kernels that begin under each other's end."""
import torch
import pytest

from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc
from tensor_matmul_collective_gb300 import decode_step as ds

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("n", [8, 40, 264])
def test_int8_weights_between_8_bit_products(n):
    R, hidden = 2, 512
    g = torch.Generator().manual_seed(7)
    w16 = [(torch.randn(hidden, hidden, generator=g) * hidden ** -0.5).to(BF).to(DEV) for _ in range(R)]
    w8 = [torch.randint(-127, 128, (hidden, hidden), generator=g, dtype=torch.int8).to(DEV) for _ in range(R)]
    s8 = [torch.full((1,), 2.0 ** -11, dtype=BF, device=DEV) for _ in range(R)]
    mlps = [ds.random_mlp(R, hidden, f, seed=f) for f in (256, 1024)]
    start = [torch.randn(n, hidden, generator=g).to(BF).to(DEV) for _ in range(R)]

    def chain(wait):
        x = start
        for _ in range(10):
            for step in (lambda x: coc.matmul_all_reduce_w8a16(x, w8, s8, "tensor"), lambda x: mlps[0](x)[0],
                         lambda x: coc.matmul_all_reduce(x, w16), lambda x: mlps[1](x)[0]):
                x = step(x)
                if wait:
                    torch.cuda.synchronize()
        return x
    want = [t.clone() for t in chain(True)]
    assert all(t.isfinite().all() for t in want)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    coc.sync_status()
