"""Append of a part of a batch: rows of the block table, lengths and offsets cut
out of a larger call's, whose first offset is a page or more."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import appended, check_append, split, to_cache

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

BATCHES = [
    # R, hq, hkv, d, rot, page, new tokens, earlier tokens, first sequence of the part, one past its last, dtype
    (1, 4, 1, 64, 64, 16, [16, 1], [0, 0], 1, 2, BF),
    (2, 8, 2, 128, 128, 64, [64, 200, 1, 3, 90], [5, 0, 63, 0, 70], 2, 5, BF),
    (1, 3, 3, 80, 40, 32, [1, 40, 0, 33, 2, 1], [30, 7, 2, 31, 0, 9], 3, 5, HF),
    (1, 2, 1, 32, 0, 16, [300, 1, 1, 1, 20], [0, 0, 15, 16, 3], 1, 4, BF),
]


@pytest.mark.parametrize("R,hq,hkv,d,rot,page,news,past,a,b,dt", BATCHES)
def test_part_of_a_batch(R, hq, hkv, d, rot, page, news, past, a, b, dt):
    lens, table, rk, rv, qkv, cos, sin = appended(R, hq, hkv, d, rot, page, news, past, dt, seed=page + d)
    part = [table[s, p].item() for s in range(a, b) for p in range(-(-lens[s] // page))]
    for codes, scale in rk + rv:            # pages of the others as they are before their first token, or with codes but no scale
        for j in range(codes.shape[0]):
            if j not in part:
                scale[j] = 0.0
    cu = kv.offsets(news)
    cache = to_cache(rk, rv)
    dev = [split(t.to(DEV), hq, hkv, d) for t in qkv]
    tb, ln, at = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    out = coc.kv_cache_append([x[1] for x in dev], [x[2] for x in dev], cache, tb[a:b], ln[a:b], None if cos is None else cos.to(DEV),
                              None if sin is None else sin.to(DEV), qs=[x[0] for x in dev], cu_new=at[a:b + 1])
    coc.sync_status()
    mine = slice(cu[a], cu[b])
    check_append(cache, [o[mine] for o in out], R, hq, hkv, d, page, news[a:b], past[a:b], lens[a:b], table[a:b], rk, rv,
                 [t[mine] for t in qkv], cos, sin, False, dt)
    for o, x in zip(out, dev):
        assert torch.equal(o[:cu[a]], x[0][:cu[a]]) and torch.equal(o[cu[b]:], x[0][cu[b]:])
