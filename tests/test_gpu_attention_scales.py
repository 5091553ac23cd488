"""Page scales of V that lie far apart: a key whose values are nothing beside
the others' still counts in the denominator."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from test_gpu_kv_cache import attend, build, check, to_cache

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

CASES = [
    # hq, hkv, d, page, new tokens, lengths, pages without values, dtype, 2-exponent of the others
    (8, 1, 128, 64, [1], [300], "first", BF, 40),
    (8, 1, 128, 64, [1], [300], "last", BF, 40),
    (4, 2, 64, 16, [1, 2], [150, 333], "even", BF, 40),
    (4, 2, 64, 16, [1, 2], [150, 333], "odd", BF, 80),
    (8, 1, 256, 128, [1], [5000], "even", BF, 30),
    (8, 1, 128, 16, [1], [30000], "first", BF, 60),         # parts of many blocks, merged
    (8, 1, 128, 16, [1], [30000], "last", BF, 60),
    (4, 1, 64, 32, [1] * 120, list(range(1, 1201, 10)), "odd", BF, 50),      # few parts an item
    (16, 1, 128, 128, [1, 1], [700, 90], "even", BF, 40),   # tiles of 16 rows
    (8, 1, 128, 64, [1], [300], "even", HF, 4),
]


@pytest.mark.parametrize("hq,hkv,d,page,news,lens,empty,dt,v_exp", CASES)
def test_pages_without_values_keep_their_weight(hq, hkv, d, page, news, lens, empty, dt, v_exp):
    table, rk, rv, qs = build(1, hq, hkv, d, page, news, lens, dt, seed=len(lens) + page, width=4096 * 64 // page if hq == 16 else None)
    codes, scale = rv[0]
    scale *= 2.0 ** v_exp
    for s, n in enumerate(lens):
        pages = -(-n // page)
        for p in range(pages):
            if {"first": p < pages // 2, "last": p >= pages // 2, "even": p % 2 == 0, "odd": p % 2 == 1}[empty]:
                codes[table[s, p].item()] = 0
                scale[table[s, p].item()] = 2.0 ** -100         # as the append leaves a page of zeros
    outs = attend(to_cache(rk, rv), table, lens, kv.offsets(news), qs)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, kv.offsets(news), page)
