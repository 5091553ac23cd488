"""Chains of the decode-step operators under dependent launches: each call
reads what the call before it has just written, and gives the bits that it
gives when it is waited for."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import to_cache

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
R, HQ, HKV, D, PAGE, B, STEPS = 2, 8, 2, 64, 16, 24, 40


def chain(wait, seed=3):
    """STEPS single-token steps: projections made of a running activation, append, attention, product, and the next
    activation; lengths move by a kernel between the steps."""
    g = torch.Generator().manual_seed(seed)
    lens0 = [1 + 7 * i for i in range(B)]
    full = [n + STEPS for n in lens0]
    table, pages = kv.make_table(full, PAGE, gen=g)
    cache = to_cache(kv.random_cache(R, pages, HKV, PAGE, D, g), kv.random_cache(R, pages, HKV, PAGE, D, g))
    tb, lens = table.to(DEV), torch.tensor(lens0, dtype=torch.int32, device=DEV)
    ang = torch.arange(max(full), dtype=torch.float64)[:, None] * 50.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    words = [torch.randint(-2 ** 31, 2 ** 31, (HQ * D // 8, HQ * D), generator=g).to(torch.int32).to(DEV) for _ in range(R)]
    scales = [torch.full((HQ * D // 64, HQ * D), 0.01, dtype=BF, device=DEV) for _ in range(R)]
    x = [torch.randn(B, HQ * D, generator=g).to(BF).to(DEV) for _ in range(R)]
    qo, ctx, y = ([torch.empty(B, HQ, D, dtype=BF, device=DEV) for _ in range(R)] for _ in range(3))
    log = []
    torch.cuda.synchronize()

    def done():
        if wait:
            torch.cuda.synchronize()
    for _ in range(STEPS):
        lens += 1
        done()
        q = [t.view(B, HQ, D) for t in x]
        coc.kv_cache_append([t[:, :HKV] for t in q], [t[:, HKV:2 * HKV] for t in q], cache, tb, lens, cos, sin, qs=q, q_outs=qo)
        done()
        coc.kv_cache_attention(qo, cache, tb, lens, outs=ctx)
        done()
        coc.matmul_all_reduce_w4a16([t.view(B, HQ * D) for t in ctx], words, scales, 64, outs=[t.view(B, HQ * D) for t in y])
        done()
        # the product's rows are the next step's activation: attention of them as they are, then back into x
        coc.kv_cache_attention(y, cache, tb, lens, outs=[t.view(B, HQ, D) for t in x])
        done()
        log.append(torch.stack([t.view(-1) for t in x + y]).clone())
        done()
    torch.cuda.synchronize()
    coc.sync_status()
    return torch.stack(log), [t.view(torch.uint8).clone() for t in cache.k + cache.v], [t.clone() for t in cache.k_scale + cache.v_scale]


def test_chain_gives_the_bits_of_calls_that_are_waited_for():
    a, b = chain(True), chain(False)
    assert torch.isfinite(a[0].float()).all()
    assert torch.equal(a[0], b[0])
    assert all(torch.equal(x, y) for x, y in zip(a[1] + a[2], b[1] + b[2]))
