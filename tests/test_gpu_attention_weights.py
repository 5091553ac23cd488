"""Softmax weights of the cached attention keep far more than 11 bits, for both
output types: values that cancel leave an output in which a weight's rounding
shows, while the output's own rounding does not."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import attend, to_cache

BF, HF = torch.bfloat16, torch.float16


def cancelling(d, hq, hkv, page, news, lens, dt, seed, width=None):
    """Keys in pairs 2 j, 2 j + 1 that differ by 2**-7 in one value, with opposite values of V.  All products of q and k are
    multiples of 2**-10 and their sums below 2**5: every logit is exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    table, pages = kv.make_table(lens, page, width=width, gen=g)
    shape = (pages, hkv, page // 2, d)
    k = torch.randint(-2, 3, shape, generator=g).double() * 0.5
    k[..., 8:] = 0                          # logits of a few units
    k = torch.stack((k, k), 3).reshape(pages, hkv, page, d).clone()
    k[:, :, 0::2, 0], k[:, :, 1::2, 0] = 0.0, 2.0 ** -7
    v = kv.e4m3(torch.randn(shape, generator=g, dtype=torch.float64))
    v = torch.stack((v, -v), 3).reshape(pages, hkv, page, d)
    one = torch.ones(pages, hkv)
    rk, rv = ([(x.float().to(kv.E4M3).view(torch.uint8), one)] for x in (k, v))
    q = (torch.randint(-8, 9, (sum(news), hq, d), generator=g).double() / 8)
    q[..., 0] = 1.0
    return table, rk, rv, [q.to(dt)]


def weight_bound(ref, size, reach, dtype):
    """The output's rounding, and weights: the logit in log2 units is at most z = 1.4427 reach; its factor is rounded three
    times (3 z 2**-24), it is added to the running reference, itself a sum of roundings (5 numbers of at most z + 15), and
    the exponential is good to 2**-22: an absolute error of (3 z + 5 (z + 15)) 2**-24 in the exponent, times ln 2, in the
    weight and once more in the sum; 2**-21 for a weight of two 11-bit halves and fp32 sums."""
    assert reach.max() <= 8
    z = 1.4427 * reach
    w = 2 * (0.7 * (8 * z + 75) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -21
    return kv.unit(dtype) * ref.abs() + w * size + 2.0 ** -24


CASES = [
    # d, hq, hkv, page, new tokens, lengths, width
    (128, 8, 1, 64, [1, 1, 1], [8, 4, 16], None),
    (64, 8, 2, 16, [1] * 5, [2, 6, 10, 32, 4], None),
    (256, 4, 1, 16, [1, 1], [8, 12], None),
    (80, 5, 1, 32, [1, 1], [6, 20], None),
    (128, 16, 1, 128, [1, 1], [8, 10], 2048),           # tiles of 16 rows
    (64, 12, 1, 64, [1, 1], [4, 12], 4096),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d,hq,hkv,page,news,lens,width", CASES)
def test_weights_keep_their_bits(d, hq, hkv, page, news, lens, width, dt):
    table, rk, rv, qs = cancelling(d, hq, hkv, page, news, lens, dt, seed=d + hq, width=width)
    outs = attend(to_cache(rk, rv), table, lens, None, qs, scale=1.0)
    coc.sync_status()
    ref, size, reach = kv.attention(qs[0], kv.values(*rk[0]), kv.values(*rv[0]), table, lens, kv.offsets(news), page, 1.0)
    err = (outs[0].cpu().double() - ref).abs()
    assert (err <= weight_bound(ref, size, reach, dt)).all(), (err / weight_bound(ref, size, reach, dt)).max()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d,hq,hkv,page,news,lens,width", CASES)
def test_the_bound_tells_11_bits(d, hq, hkv, page, news, lens, width, dt):
    """The same inputs with weights rounded to 11 bits in the oracle lie outside the bound."""
    table, rk, rv, qs = cancelling(d, hq, hkv, page, news, lens, dt, seed=d + hq, width=width)
    k, v = kv.values(*rk[0]), kv.values(*rv[0])
    ref, size, reach = kv.attention(qs[0], k, v, table, lens, kv.offsets(news), page, 1.0)
    worst = 0.0
    for s, n in enumerate(lens):
        kk, vv = kv.gather(k, table[s], n, page), kv.gather(v, table[s], n, page)
        z = qs[0][s].double().view(hkv, hq // hkv, d) @ kk.transpose(1, 2)
        w = torch.exp(z - z.amax(2, keepdim=True))
        rounded = (w * 512).to(torch.float16).double() / 512
        out = ((rounded @ vv) / w.sum(2, keepdim=True)).view(hq, d).to(dt).double()
        worst = max(worst, ((out - ref[s]).abs() / weight_bound(ref, size, reach, dt)[s]).max().item())
    assert worst > 2
