"""New tokens that belong to no sequence: the padding of a batch of fixed size."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import APPEND, appended, attend, build, check, check_append, split, to_cache

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def dev32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("hq", [0, 6])
def test_append_of_a_padded_batch(hq):
    """Rotation tables of exactly the lengths: tokens past the last offset have no position, q is copied, nothing is reported."""
    R, hkv, d, rot, page, news, past = 2, 2, 64, 64, 32, [3, 1], [30, 7]
    lens, table, rk, rv, qkv, cos, sin = appended(R, hq, hkv, d, rot, page, news, past, BF, seed=3)
    cos, sin = cos[:max(lens)].contiguous(), sin[:max(lens)].contiguous()
    g = torch.Generator().manual_seed(4)
    padded = [torch.cat((t, torch.randn(40, t.shape[1], generator=g).to(BF))) for t in qkv]
    cache = to_cache(rk, rv)
    dev = [split(t.to(DEV), hq, hkv, d) for t in padded]
    out = coc.kv_cache_append([x[1] for x in dev], [x[2] for x in dev], cache, table.to(DEV), dev32(lens), cos.to(DEV), sin.to(DEV),
                              qs=[x[0] for x in dev] if hq else None, cu_new=dev32(kv.offsets(news)))
    coc.sync_status()
    check_append(cache, [o[:4] for o in out] if hq else out, R, hq, hkv, d, page, news, past, lens, table, rk, rv, qkv, cos, sin, False, BF)
    for o, x in zip(out or [], dev):
        assert torch.equal(o[4:], x[0][4:])


@pytest.mark.parametrize("R,hq,hkv,d,dt", [(2, 8, 2, 64, BF), (1, 5, 1, 80, HF), (1, 24, 2, 16, BF)])
@pytest.mark.parametrize("news,first,pad", [([2, 1], 0, 5), ([2, 0, 1], 3, 0), ([1, 4], 70, 300), ([0, 0], 2, 9)])
def test_attention_rows_of_no_sequence_are_zero(R, hq, hkv, d, dt, news, first, pad):
    page, lens = 32, [90, 40, 33][:len(news)]
    table, rk, rv, qs = build(R, hq, hkv, d, page, news, lens, dt, seed=6)
    T = first + sum(news) + pad
    g = torch.Generator().manual_seed(7)
    wide = [torch.cat((torch.randn(first, hq, d, generator=g).to(dt), q, torch.randn(pad, hq, d, generator=g).to(dt))) for q in qs]
    outs = [torch.full((T, hq, d), float("nan"), dtype=dt, device=DEV) for _ in range(R)]
    cu = [first + c for c in kv.offsets(news)]
    attend(to_cache(rk, rv), table, lens, cu, wide, outs=outs)
    coc.sync_status()
    end = first + sum(news)
    for o in outs:
        assert not o[:first].any() and not o[end:].any()
    check([o[first:end] for o in outs], qs, rk, rv, table, lens, kv.offsets(news), page)
