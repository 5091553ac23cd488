"""New outputs of a call on another stream: their memory is that stream's, not
what the current stream has freed and its kernels still use."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc
from tensor_matmul_collective_gb300 import decode_step as ds

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import build, to_cache

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, HQ, D = 64, 16, 256


def calls():
    table, rk, rv, qs = build(1, HQ, 2, D, 16, [1] * B, [20] * B, BF, seed=1)
    cache, tb, q = to_cache(rk, rv), table.to(DEV), [x.to(DEV) for x in qs]
    lens = torch.full((B,), 20, dtype=torch.int32, device=DEV)
    words = [torch.zeros(HQ * D // 8, HQ * D, dtype=torch.int32, device=DEV)]
    scales = [torch.ones(HQ * D // 128, HQ * D, dtype=BF, device=DEV)]
    k = [x[:, :2] for x in q]
    return {"append": lambda s: coc.kv_cache_append(k, k, cache, tb, lens, qs=q, stream=s),
            "attend": lambda s: coc.kv_cache_attention(q, cache, tb, lens, stream=s),
            "w4": lambda s: coc.matmul_all_reduce_w4a16([q[0].view(B, HQ * D)], words, scales, 128, stream=s)}


def freed_and_read(f):
    """What a kernel of the current stream reads from a tensor that was freed behind it, while f runs elsewhere."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(B, HQ, D, dtype=BF, device=DEV)
    old = torch.full((B, HQ, D), 7.0, dtype=BF, device=DEV)
    torch.cuda._sleep(200_000_000)
    kept.copy_(old)
    del old
    f()
    torch.cuda.synchronize()
    return kept


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("name", ["append", "attend", "w4"])
@pytest.mark.parametrize("handle", [False, True])
def test_new_outputs_are_the_streams(monkeypatch, native, name, handle):
    if not native:
        monkeypatch.setattr(coc, "_native", False)
        monkeypatch.setattr(coc, "_marshal", lambda: False)
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)[0].clone()
    call(side)
    got = []

    def f():
        got.append(call(side.cuda_stream if handle else side)[0])
        side.synchronize()
    assert (freed_and_read(f) == 7).all()
    assert torch.equal(got[0], want)
    coc.sync_status()


def test_a_block_on_another_stream():
    """All that a block allocates on the way is the stream's too."""
    block = ds.random_block(1, 512, 8, 2, 64, pages=B, page_size=16, positions=16, seed=2)
    table = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    x = [torch.randn(B, 512, device=DEV).to(BF)]
    side = torch.cuda.Stream()
    want = block(x, table, lens)[0].clone()
    torch.cuda.synchronize()
    block(x, table, lens, stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    shapes = [(B, 512), (B, 12 * 64), (B, 8, 64), (B, 8, 64)]
    kept = [torch.empty(s, dtype=BF, device=DEV) for s in shapes]
    old = [torch.full(s, 7.0, dtype=BF, device=DEV) for s in shapes]
    torch.cuda._sleep(200_000_000)
    for a, b in zip(kept, old):
        a.copy_(b)
    del a, b, old
    got = block(x, table, lens, stream=side)[0]
    side.synchronize()
    torch.cuda.synchronize()
    assert all((a == 7).all() for a in kept)
    assert torch.equal(got, want)
    coc.sync_status()
