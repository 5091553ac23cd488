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


def test_every_lane_has_the_scale_from_before():
    """A warp a unit, each new token far above what its page holds: all codes of the page shrink by the same factor, none by 1."""
    page, d, hkv, seqs = 16, 256, 2, 200
    g = torch.Generator().manual_seed(5)
    lens = [2 + s % 15 for s in range(seqs)]
    table, pages = kv.make_table(lens, page, gen=g)
    rk, rv = kv.random_cache(1, pages, hkv, page, d, g), kv.random_cache(1, pages, hkv, page, d, g)
    new = [(8.0 * torch.randn(seqs, hkv, d, generator=g)).to(BF)]
    cache = to_cache(rk, rv)
    coc.kv_cache_append([new[0].to(DEV)], [new[0].to(DEV)], cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    coc.sync_status()
    for (codes0, scale0), codes1, scale1 in ((rk[0], cache.k[0], cache.k_scale[0]), (rv[0], cache.v[0], cache.v_scale[0])):
        grown = 0
        for s, n in enumerate(lens):
            j = table[s, 0].item()
            f = scale0[j].double() / scale1[j].cpu().double()
            grown += int((f < 1).sum())
            old = codes0[j, :, :n - 1].view(kv.E4M3).double() * f[:, None, None]
            assert torch.equal(codes1[j, :, :n - 1].float().cpu().double(), kv.e4m3(old))
        assert grown > seqs
