"""The paged 8-bit key/value cache on the GPU: append (rotation, page scales,
codes) and attention over it, against plain float64 definitions, at the
lengths, pages, windows and layouts where they can go wrong."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def to_cache(ranks_k, ranks_v):
    def up(u8):
        return u8.to(DEV).view(kv.E4M3)
    return coc.KVCache([up(c) for c, _ in ranks_k], [up(c) for c, _ in ranks_v], [s.to(DEV) for _, s in ranks_k],
                       [s.to(DEV) for _, s in ranks_v])


# ---------------------------------------------------------------- attention ---

def build(R, hq, hkv, d, page, news, lens, dt, seed, q_std=1.5, width=None):
    g = torch.Generator().manual_seed(seed)
    table, pages = kv.make_table(lens, page, width=width, gen=g)
    rk, rv = kv.random_cache(R, pages, hkv, page, d, g), kv.random_cache(R, pages, hkv, page, d, g)
    T = sum(news)
    qs = [(q_std * torch.randn(T, hq, d, generator=g)).to(dt) for _ in range(R)]
    return table, rk, rv, qs


def attend(cache, table, lens, cu, qs, **kw):
    return coc.kv_cache_attention([q.to(DEV) if q.device != DEV else q for q in qs], cache, table.to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV),
                                  cu_new=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV), **kw)


def check(outs, qs, rk, rv, table, lens, cu, page, window=0, sinks=0, scale=None):
    d = qs[0].shape[2]
    for r, o in enumerate(outs):
        ref, size, reach = kv.attention(qs[r], kv.values(*rk[r]), kv.values(*rv[r]), table, lens, cu, page,
                                        d ** -0.5 if scale is None else scale, window, sinks)
        got = o.cpu().double()
        err = (got - ref).abs()
        bound = kv.attention_bound(ref, size, reach, max(lens, default=0), qs[r].dtype)
        assert torch.isfinite(got).all()
        bad = (err > bound).nonzero()
        assert not len(bad), f"rank {r}: {len(bad)} outside, first {bad[0].tolist()}: {got[tuple(bad[0])]} for {ref[tuple(bad[0])]}"


CASES = [
    # R, hq, hkv, d, page, new tokens, lengths, window, sinks, dtype
    (1, 8, 1, 128, 64, [1], [1], 0, 0, BF),
    (1, 1, 1, 16, 16, [1], [17], 0, 0, HF),
    (2, 4, 4, 64, 16, [1, 1, 1], [15, 16, 33], 0, 0, BF),
    (1, 32, 8, 128, 64, [1, 1], [777, 64], 0, 0, HF),
    (8, 8, 1, 128, 128, [1] * 5, [0, 1, 129, 500, 128], 0, 0, BF),
    (1, 5, 1, 80, 32, [2, 0, 3, 1], [100, 50, 2, 31], 0, 0, HF),      # rows that see nothing: 3 new tokens, 2 positions
    (2, 12, 4, 96, 64, [4, 1, 7], [4, 300, 130], 0, 0, BF),           # whole prompts and continuations
    (1, 9, 3, 112, 16, [1, 2], [200, 75], 0, 0, BF),
    (1, 16, 2, 256, 64, [1, 3], [321, 3], 0, 0, BF),
    (1, 2, 2, 192, 32, [5], [97], 0, 0, HF),
    (1, 40, 2, 64, 64, [1, 1], [1000, 40], 0, 0, HF),                 # 20 query heads share a key head
    (1, 8, 1, 128, 64, [1, 1, 1], [1000, 63, 5], 100, 4, BF),         # window and sinks far apart, near, all
    (1, 4, 2, 64, 16, [3, 2], [210, 17], 1, 0, HF),                   # a window of the token itself
    (2, 8, 2, 128, 32, [6, 1], [500, 499], 33, 70, BF),               # more sinks than a page
    (1, 8, 8, 48, 128, [1, 9], [257, 640], 64, 1, HF),
    (1, 8, 1, 128, 64, [70], [200], 0, 0, BF),                        # many new tokens
    (1, 6, 2, 128, 16, [33, 1], [33, 4000], 0, 0, HF),
]


@pytest.mark.parametrize("R,hq,hkv,d,page,news,lens,window,sinks,dt", CASES)
def test_attention(R, hq, hkv, d, page, news, lens, window, sinks, dt):
    table, rk, rv, qs = build(R, hq, hkv, d, page, news, lens, dt, seed=hash((hq, d, page)) % 1000)
    cu = kv.offsets(news)
    cache = to_cache(rk, rv)
    outs = attend(cache, table, lens, cu, qs, window=window, sinks=sinks)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, cu, page, window, sinks)
    if all(n == 1 for n in news):
        again = attend(cache, table, lens, None, qs, window=window, sinks=sinks)
        assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("B,length,hkv", [(1, 40000, 1), (3, 9001, 2), (130, 300, 1), (400, 37, 2)])
def test_attention_work_split(B, length, hkv):
    """Few long sequences (split over many blocks) and many short ones, lengths all different; twice the same bits."""
    lens = [max(1, length - 7 * i) for i in range(B)]
    table, rk, rv, qs = build(1, 4 * hkv, hkv, 64, 64, [1] * B, lens, BF, seed=B)
    cache = to_cache(rk, rv)
    outs = attend(cache, table, lens, None, qs)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, kv.offsets([1] * B), 64)
    again = attend(cache, table, lens, None, qs)
    assert torch.equal(outs[0], again[0])


@pytest.mark.parametrize("seed,q_std,k_exp,v_exp", [(1, 30.0, 0, 0), (2, 1e-3, 0, 0), (3, 1.0, -40, 30), (4, 1.0, 0, -60), (5, 6e4, -20, 0)])
def test_attention_ranges(seed, q_std, k_exp, v_exp):
    """Peaked and flat softmax, keys and values of other magnitudes (their scales carry them), q near bf16 sizes fp16 lacks."""
    news, lens = [1, 2], [150, 333]
    dt = BF
    table, rk, rv, qs = build(1, 8, 2, 128, 32, news, lens, dt, seed, q_std=q_std)
    rk = [(c, s * 2.0 ** k_exp) for c, s in rk]
    rv = [(c, s * 2.0 ** v_exp) for c, s in rv]
    scale = 128 ** -0.5 * 2.0 ** -k_exp / (q_std if q_std > 100 else 1.0)
    outs = attend(to_cache(rk, rv), table, lens, kv.offsets(news), qs, scale=scale)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, kv.offsets(news), 32, scale=scale)


def test_attention_pages_of_unlike_scales():
    """One page whose values are 2**20 times the others' and one that is all zero."""
    news, lens = [1], [300]
    table, rk, rv, qs = build(1, 4, 1, 64, 32, news, lens, BF, seed=9)
    for ranks, at, f in ((rv, 3, 2.0 ** 20), (rv, 4, 2.0 ** -30), (rk, 5, 4.0)):
        ranks[0][1][table[0, at].item()] *= f
    z = table[0, 6].item()
    rv[0][0][z] = 0
    rv[0][1][z] = 2.0 ** -100
    outs = attend(to_cache(rk, rv), table, lens, [0, 1], qs)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, [0, 1], 32)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
def test_attention_nothing_unseen_comes_in(window, sinks):
    """NaN codes past the lengths, in pages of nobody and (with a window) in positions no row sees; scales of unused pages NaN."""
    page, news, lens = 32, [2, 1, 1], [70, 129, 32]
    table, rk, rv, qs = build(1, 8, 2, 128, page, news, lens, BF, seed=4)
    used = set()
    for s, n in enumerate(lens):
        for p in range(-(-n // page)):
            used.add(table[s, p].item())
    clean = ([(rk[0][0].clone(), rk[0][1])], [(rv[0][0].clone(), rv[0][1])])
    seen = {s: set().union(*[set(kv.visible(lens[s] - i, window, sinks)) for i in range(news[s])]) for s in range(3)}
    for codes, scale in (rk[0], rv[0]):
        for i in range(codes.shape[0]):
            if i not in used:
                codes[i] = kv.NAN_CODE
                scale[i] = float("nan")
        for s, n in enumerate(lens):
            for p in range(-(-n // page) * page):
                if p not in seen[s]:
                    codes[table[s, p // page].item(), :, p % page] = kv.NAN_CODE
    outs = attend(to_cache(rk, rv), table, lens, kv.offsets(news), qs, window=window, sinks=sinks)
    coc.sync_status()
    check(outs, qs, *clean, table, lens, kv.offsets(news), page, window, sinks)


@pytest.mark.parametrize("d,hq", [(128, 8), (64, 2), (256, 4)])
def test_attention_nan_reaches_only_rows_that_see_it(d, hq):
    """A NaN value of the second of three new tokens: the first token's rows are clean, the others have NaN in that value only.
    A NaN key of the last token: only the last token's rows are NaN."""
    news, lens = [3], [50]
    table, rk, rv, qs = build(1, hq, 1, d, 16, news, lens, BF, seed=5)
    c = rv[0][0]
    page48 = table[0, 3].item()
    clean_v = [(c.clone(), rv[0][1])]
    c[page48, 0, 0, 7] = kv.NAN_CODE             # position 48: seen by new tokens 1 and 2
    outs = attend(to_cache(rk, rv), table, lens, [0, 3], qs)
    coc.sync_status()
    got = outs[0].cpu().double()
    assert torch.isfinite(got[0]).all()
    assert torch.isnan(got[1:, :, 7]).all()
    rest = [i for i in range(d) if i != 7]
    ref, size, reach = kv.attention(qs[0], kv.values(*rk[0]), kv.values(*clean_v[0]), table, lens, [0, 3], 16, d ** -0.5)
    bound = kv.attention_bound(ref, size, reach, 50, BF)
    assert ((got - ref).abs() <= bound)[:, :, rest].all()
    assert ((got - ref).abs() <= bound)[0].all()
    rk[0][0][page48, 0, 1, 3] = kv.NAN_CODE      # position 49: seen by new token 2 alone
    outs = attend(to_cache(rk, clean_v), table, lens, [0, 3], qs)
    got = outs[0].cpu().double()
    assert torch.isnan(got[2]).all()
    assert ((got - ref).abs() <= bound)[:2].all()


def test_attention_strided_q_and_given_outputs():
    news, lens = [2, 1], [90, 40]
    table, rk, rv, qs = build(2, 8, 2, 64, 32, news, lens, HF, seed=6)
    wide = [torch.zeros(3, 20, 64, dtype=HF) for _ in qs]
    for w, q in zip(wide, qs):
        w[:, 2:18:2] = q
    dev = [w.to(DEV)[:, 2:18:2] for w in wide]
    outs = [torch.full((3, 8, 64), float("nan"), dtype=HF, device=DEV) for _ in qs]
    got = attend(to_cache(rk, rv), table, lens, kv.offsets(news), dev, outs=outs)
    coc.sync_status()
    assert got[0] is outs[0] and got[1] is outs[1]
    check(outs, qs, rk, rv, table, lens, kv.offsets(news), 32)


def test_attention_bad_pages_are_left_out_and_reported():
    news, lens = [1, 1], [100, 64]
    table, rk, rv, qs = build(1, 4, 1, 64, 32, news, lens, BF, seed=7)
    bad = table.clone()
    bad[0, 1] = 10 ** 6
    cache = to_cache(rk, rv)
    outs = attend(cache, bad, lens, None, qs)
    with pytest.raises(coc.CocError) as e:
        coc.sync_status()
    assert e.value.status == coc.ERR_INVALID_ARG and "KV cache" in e.value.detail
    coc.sync_status()
    k, v = kv.values(*rk[0]), kv.values(*rv[0])
    ids = torch.cat([torch.arange(32), torch.arange(64, 100)])
    kk, vv = kv.gather(k, table[0], 100, 32)[:, ids], kv.gather(v, table[0], 100, 32)[:, ids]
    ref = torch.softmax(qs[0][0].double().view(1, 4, 64) @ kk.transpose(1, 2) * 64 ** -0.5, 2) @ vv
    assert (outs[0][0].cpu().double() - ref[0]).abs().max() < 0.02
    # a length beyond the table: the positions there are left out
    outs = attend(cache, table[:, :2].contiguous(), lens, None, qs)
    with pytest.raises(coc.CocError):
        coc.sync_status()
    check([o[1:] for o in outs], [q[1:] for q in qs], rk, rv, table[1:], [64], [0, 1], 32)


def test_attention_beyond_4_gib_of_codes():
    """Pages past byte offset 2**32 (and element offset 2**31) of the code buffers."""
    page, d, H = 128, 128, 2
    pages = (1 << 32) // (page * d * H) + 3
    g = torch.Generator().manual_seed(8)
    small = kv.random_cache(1, 3, H, page, d, g), kv.random_cache(1, 3, H, page, d, g)
    big = []
    for ranks in small:
        c = torch.zeros(pages, H, page, d, dtype=torch.uint8, device=DEV)
        s = torch.ones(pages, H, dtype=torch.float32, device=DEV)
        c[-3:], s[-3:] = ranks[0][0].to(DEV), ranks[0][1].to(DEV)
        big.append((c.view(kv.E4M3), s))
    cache = coc.KVCache([big[0][0]], [big[1][0]], [big[0][1]], [big[1][1]])
    q = [torch.randn(1, 4, d, generator=g).to(BF)]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    outs = attend(cache, table + (pages - 3), [300], None, q)
    coc.sync_status()
    check(outs, q, small[0], small[1], table, [300], [0, 1], page)
    # and an append there
    k, v = [torch.randn(1, H, d, generator=g).to(BF)], [torch.randn(1, H, d, generator=g).to(BF)]
    coc.kv_cache_append([x.to(DEV) for x in k], [x.to(DEV) for x in v], cache, (table + (pages - 3)).to(DEV),
                        torch.tensor([384], dtype=torch.int32, device=DEV))
    coc.sync_status()
    got = big[0][0].view(torch.uint8)[pages - 3 + 1, :, 127].cpu().view(kv.E4M3).double() * big[0][1][pages - 2].cpu().double()[:, None]
    assert ((got - k[0][0].double()).abs() <= 0.0625 * k[0][0].double().abs() + 0.01).all()


def test_attention_streams_and_graphs():
    """On a side stream behind the work that makes its inputs, and captured: replays follow new inputs."""
    news, lens = [1] * 4, [500, 20, 3000, 129]
    table, rk, rv, qs = build(1, 8, 1, 128, 64, news, lens, BF, seed=11)
    cache = to_cache(rk, rv)
    tb, ln = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = [x.to(DEV) for x in qs]
    want = coc.kv_cache_attention(q, cache, tb, ln)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(8):
            big = big @ big * 1e-3
        late = [x.clone() + (big[0, 0] * 0).nan_to_num().to(BF) for x in q]
        got = coc.kv_cache_attention(late, cache, tb, ln)[0]
    side.synchronize()
    assert torch.equal(got, want)
    static = [x.clone() for x in q]
    outs = [torch.empty_like(q[0])]
    with torch.cuda.stream(side):
        coc.kv_cache_attention(static, cache, tb, ln, outs=outs)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        coc.kv_cache_attention(static, cache, tb, ln, outs=outs)
    for f in (1.0, -0.5):
        static[0].copy_(q[0] * f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], coc.kv_cache_attention([q[0] * f], cache, tb, ln)[0])
    coc.sync_status()


# ------------------------------------------------------------------- append ---

def rotate64(x, pos, cos, sin, interleaved):
    """(rotated, size of the terms) in float64."""
    half = cos.shape[1]
    out, size = x.double().clone(), x.double().abs()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
    xa, xb = x.double()[:, :, a], x.double()[:, :, b]
    out[:, :, a], out[:, :, b] = xa * c - xb * s, xb * c + xa * s
    size[:, :, a] = (xa * c).abs() + (xb * s).abs()
    size[:, :, b] = (xb * c).abs() + (xa * s).abs()
    return out, size


APPEND = [
    # R, hq, hkv, d, rot, page, new tokens, earlier tokens, interleaved, dtype
    (1, 8, 1, 128, 128, 64, [1], [0], False, BF),
    (1, 2, 2, 16, 16, 16, [1, 1], [15, 16], True, HF),
    (8, 8, 1, 128, 128, 64, [1] * 6, [5, 63, 64, 0, 100, 127], False, BF),
    (2, 6, 3, 80, 40, 32, [3, 0, 50, 1], [30, 7, 20, 31], False, HF),
    (1, 4, 4, 96, 96, 128, [300, 129], [0, 100], True, BF),
    (1, 5, 1, 256, 64, 16, [17, 40, 2], [3, 16, 14], False, BF),
    (2, 0, 2, 64, 0, 64, [100, 1], [1, 63], False, HF),                # no q, no rotation
    (1, 3, 1, 48, 6, 32, [2, 33], [62, 31], True, BF),                 # a rotation of 6 values
    (1, 1, 1, 192, 190, 64, [5], [60], False, HF),
]


def appended(R, hq, hkv, d, rot, page, news, past, dt, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(news, past)]
    table, pages = kv.make_table(lens, page, gen=g)
    rk, rv = kv.random_cache(R, pages, hkv, page, d, g), kv.random_cache(R, pages, hkv, page, d, g)
    T = sum(news)
    width = (hq + 2 * hkv) * d
    qkv = [(gain * torch.randn(T, width, generator=g)).to(dt) for _ in range(R)]
    cos = sin = None
    if rot:
        ang = torch.arange(max(lens) + 3, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))
        cos, sin = ang.cos().float(), ang.sin().float()
    return lens, table, rk, rv, qkv, cos, sin


def split(t, hq, hkv, d):
    T = t.shape[0]
    return t[:, :hq * d].view(T, hq, d), t[:, hq * d:(hq + hkv) * d].view(T, hkv, d), t[:, (hq + hkv) * d:].view(T, hkv, d)


def check_append(cache, q_outs, R, hq, hkv, d, page, news, past, lens, table, rk, rv, qkv, cos, sin, interleaved, dt):
    cu = kv.offsets(news)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(past, news)])
    for r in range(R):
        q, k, v = split(qkv[r], hq, hkv, d)
        if hq:
            ref, size = rotate64(q, pos, cos, sin, interleaved) if cos is not None else (q.double(), q.double().abs())
            err = (q_outs[r].cpu().double() - ref).abs()
            assert (err <= kv.unit(dt) * ref.abs() + 2.0 ** -22 * size + 2.0 ** -25).all()
        for src, (codes0, scale0), codes1, scale1, turn in ((k, rk[r], cache.k[r], cache.k_scale[r], cos is not None),
                                                           (v, rv[r], cache.v[r], cache.v_scale[r], False)):
            x, size = rotate64(src, pos, cos, sin, interleaved) if turn else (src.double(), src.double().abs())
            got, s1 = codes1.view(torch.uint8).cpu(), scale1.cpu().double()
            val = got.view(kv.E4M3).double()
            touched = torch.zeros(codes0.shape[:3], dtype=torch.bool)
            pages_seen = set()
            for s, n in enumerate(lens):
                for p in range(past[s] // page, -(-n // page)) if news[s] else []:
                    j = table[s, p].item()
                    pages_seen.add(j)
                    a, b = max(past[s], p * page), min(n, (p + 1) * page)
                    t = slice(cu[s] + a - past[s], cu[s] + b - past[s])
                    kept = a - p * page
                    for h in range(hkv):
                        S = s1[j, h].item()
                        top = x[t, h].abs().max().item()
                        want = {max(kv.page_scale(top * f), scale0[j, h].item() if kept else 0.0) for f in (1 - 2.0 ** -22, 1 + 2.0 ** -22)}
                        assert S in want, (S, want)
                        old = codes0[j, h, :kept].view(kv.E4M3).double()
                        assert torch.equal(val[j, h, :kept], kv.e4m3(old * (scale0[j, h].item() / S)))
                        y = x[t, h] / S
                        _, e = torch.frexp(y.abs())
                        ulp = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
                        err = (val[j, h, kept:kept + b - a] - y).abs()
                        assert (err <= 0.5 * ulp * (1 + 2.0 ** -20) + 2.0 ** -22 * size[t, h] / S).all()
                        touched[j, h, :kept + b - a] = True
            assert torch.equal(got[~touched], codes0[~touched])          # nothing else is written
            rest = [j for j in range(codes0.shape[0]) if j not in pages_seen]
            assert torch.equal(scale1.cpu()[rest], scale0[rest])


@pytest.mark.parametrize("gain", [1.0, 40.0, 1e-3])
@pytest.mark.parametrize("R,hq,hkv,d,rot,page,news,past,interleaved,dt", APPEND)
def test_append(R, hq, hkv, d, rot, page, news, past, interleaved, dt, gain):
    lens, table, rk, rv, qkv, cos, sin = appended(R, hq, hkv, d, rot, page, news, past, dt, seed=hq + d + page, gain=gain)
    cache = to_cache(rk, rv)
    dev = [split(t.to(DEV), hq, hkv, d) for t in qkv]
    args = ([x[1] for x in dev], [x[2] for x in dev], cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
            None if cos is None else cos.to(DEV), None if sin is None else sin.to(DEV))
    kw = dict(qs=[x[0] for x in dev] if hq else None, interleaved=interleaved,
              cu_new=torch.tensor(kv.offsets(news), dtype=torch.int32, device=DEV))
    q_outs = coc.kv_cache_append(*args, **kw)
    coc.sync_status()
    check_append(cache, q_outs, R, hq, hkv, d, page, news, past, lens, table, rk, rv, qkv, cos, sin, interleaved, dt)
    # the same tokens again leave the cache as it is
    before = [t.view(torch.uint8).clone() for t in cache.k + cache.v] + [t.clone() for t in cache.k_scale + cache.v_scale]
    coc.kv_cache_append(*args, **kw)
    after = [t.view(torch.uint8) for t in cache.k + cache.v] + cache.k_scale + cache.v_scale
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_append_special_values():
    """Zeros, NaN and infinities, the type's largest and least values; and a page whose scale grows at every step."""
    page, d = 16, 32
    cache = coc.KVCache.empty(1, 3, page, 1, d)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    k = torch.zeros(1, 1, d, dtype=BF, device=DEV)
    one = lambda n: torch.tensor([n], dtype=torch.int32, device=DEV)  # noqa: E731
    coc.kv_cache_append([k], [k], cache, table, one(1))
    assert cache.k_scale[0][1, 0].item() == 2.0 ** -100 and not cache.k[0].view(torch.uint8).any()
    x = k.clone()
    x[0, 0, :6] = torch.tensor([1.75, -0.875, float("inf"), float("-inf"), float("nan"), 0.0])
    coc.kv_cache_append([x], [x], cache, table, one(2))
    assert cache.v_scale[0][1, 0].item() == 2.0 ** -8                  # 1.75 = 448 x 2**-8
    got = cache.v[0][1, 0, 1, :6].float().cpu()
    assert got[:4].tolist() == [448.0, -224.0, 448.0, -448.0] and got[4].isnan() and got[5] == 0
    top = torch.finfo(BF).max
    x = k.clone()
    x[0, 0, 0] = top
    x[0, 0, 1] = torch.finfo(BF).smallest_normal
    coc.kv_cache_append([x], [x], cache, table, one(3))
    s = cache.k_scale[0][1, 0].item()
    assert s == kv.page_scale(top) and cache.k[0][1, 0, 2, 0].float().item() == kv.e4m3(torch.tensor(top / s, dtype=torch.float64)).item()
    assert cache.k[0][1, 0, 1, :4].float().cpu()[:2].tolist() == [0.0, 0.0]   # underflow of what is so much smaller
    coc.sync_status()
    grow = coc.KVCache.empty(1, 1, page, 1, d)
    t0 = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    for i in range(page):
        x = torch.full((1, 1, d), 2.0 ** (i - 8), dtype=BF, device=DEV)
        coc.kv_cache_append([x], [x], grow, t0, one(i + 1))
    want = torch.tensor([2.0 ** (i - 8) for i in range(page)])
    vals = grow.k[0][0, 0, :, 0].float().cpu() * grow.k_scale[0][0, 0].cpu()
    small = grow.k_scale[0][0, 0].item() * 2.0 ** -9                   # the least e4m3 value at the last scale
    assert torch.equal(vals[want >= small], want[want >= small])


def test_append_out_of_range_is_left_out_and_reported():
    page, d = 16, 32
    cache = coc.KVCache.empty(1, 2, page, 1, d)
    x = torch.ones(3, 1, d, dtype=BF, device=DEV)
    table = torch.tensor([[0], [7], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 3, 17], dtype=torch.int32, device=DEV)     # the second's page, the third's position: out of range
    q = coc.kv_cache_append([x], [x], cache, table, lens, qs=[2 * x])
    with pytest.raises(coc.CocError) as e:
        coc.sync_status()
    assert e.value.status == coc.ERR_INVALID_ARG
    codes = cache.k[0].view(torch.uint8)
    assert codes[0, 0, 2].all() and codes.count_nonzero() == d
    assert torch.equal(q[0], 2 * x)
    cos = torch.ones(2, d // 2, device=DEV)                            # position 2 has no row in the tables
    coc.kv_cache_append([x[:1]], [x[:1]], cache, table[:1], lens[:1], cos, cos)
    with pytest.raises(coc.CocError):
        coc.sync_status()
    # negative positions (fewer cached than new tokens) are left out without an error
    cache = coc.KVCache.empty(1, 2, page, 1, d)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    coc.kv_cache_append([x], [x], cache, table[:1], torch.tensor([1], dtype=torch.int32, device=DEV), cu_new=cu)
    coc.sync_status()
    assert cache.k[0].view(torch.uint8).count_nonzero() == d and cache.k[0].view(torch.uint8)[0, 0, 0].all()


def test_append_then_attend():
    """Prompts appended at once, then tokens one at a time: the attention of what the cache then holds."""
    R, hq, hkv, d, page = 2, 8, 2, 64, 32
    news, past = [45, 3], [0, 0]
    lens, table, _, _, qkv, cos, sin = appended(R, hq, hkv, d, d, page, [52, 10], past, BF, seed=3)
    cache = coc.KVCache.empty(R, 8, page, hkv, d)
    table = torch.tensor([[5, 2], [7, 0]], dtype=torch.int32)
    cos, sin = cos.to(DEV), sin.to(DEV)
    starts, ends = [0, 52], [45, 55]
    rows = torch.cat([torch.arange(a, b) for a, b in zip(starts, ends)])
    step = [split(t[rows].to(DEV), hq, hkv, d) for t in qkv]
    lens = [45, 3]
    cu = kv.offsets([45, 3])
    for i in range(8):
        ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cd = torch.tensor(cu, dtype=torch.int32, device=DEV)
        q = coc.kv_cache_append([x[1] for x in step], [x[2] for x in step], cache, table.to(DEV), ln, cos, sin,
                                qs=[x[0] for x in step], cu_new=cd)
        outs = coc.kv_cache_attention(q, cache, table.to(DEV), ln, cu_new=cd)
        coc.sync_status()
        rk = [(cache.k[r].view(torch.uint8).cpu(), cache.k_scale[r].cpu()) for r in range(R)]
        rv = [(cache.v[r].view(torch.uint8).cpu(), cache.v_scale[r].cpu()) for r in range(R)]
        check(outs, [x.cpu() for x in q], rk, rv, table, lens, cu, page)
        if i == 7:
            break
        rows = torch.tensor([lens[0], 52 + lens[1]])
        step = [split(t[rows].to(DEV), hq, hkv, d) for t in qkv]
        lens, cu = [n + 1 for n in lens], [0, 1, 2]


# ----------------------------------------------------------------- the binding ---

def test_binding_native_and_plain_marshalling_agree(monkeypatch):
    """The compiled argument marshalling and the one in Python make the same calls."""
    news, lens = [2, 1], [90, 40]
    table, rk, rv, qs = build(2, 8, 2, 64, 32, news, lens, BF, seed=21)
    tb, ln = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor(kv.offsets(news), dtype=torch.int32, device=DEV)
    q = [x.to(DEV) for x in qs]
    k = [torch.randn(3, 2, 64, device=DEV).to(BF) for _ in range(2)]
    cos = torch.rand(100, 32, device=DEV)
    got = []
    for native in (True, False):
        if not native:
            monkeypatch.setattr(coc, "_native", False)
            monkeypatch.setattr(coc, "_marshal", lambda: False)
        else:
            assert coc._marshal(), "the compiled marshalling was not built"
        cache = to_cache(rk, rv)
        turned = coc.kv_cache_append(k, k, cache, tb, ln, cos, cos, qs=q, cu_new=cu)
        outs = coc.kv_cache_attention(turned, cache, tb, ln, cu_new=cu, window=50, sinks=2)
        w = coc.matmul_all_reduce_w4a16([x.view(3, 512) for x in outs], [torch.full((64, 24), 0x12345678, dtype=torch.int32, device=DEV)] * 2,
                                        [torch.ones(4, 24, dtype=BF, device=DEV)] * 2, 128)
        got.append([*turned, *outs, *w, *[t.view(torch.uint8) for t in cache.k + cache.v], *cache.k_scale])
    coc.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("native", [True, False])
def test_binding_refusals(monkeypatch, native):
    if not native:
        monkeypatch.setattr(coc, "_native", False)
        monkeypatch.setattr(coc, "_marshal", lambda: False)
    cache = coc.KVCache.empty(2, 4, 16, 2, 64)
    x = [torch.zeros(3, 2, 64, dtype=BF, device=DEV) for _ in range(2)]
    q = [torch.zeros(3, 4, 64, dtype=BF, device=DEV) for _ in range(2)]
    tb = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    ln = torch.ones(3, dtype=torch.int32, device=DEV)
    cos = torch.zeros(4, 32, device=DEV)

    def bad(err, f, *a, **kw):
        with pytest.raises(err):
            f(*a, **kw)
    ap, at = coc.kv_cache_append, coc.kv_cache_attention
    bad(ValueError, ap, x[:1], x, cache, tb, ln)                             # ranks
    bad(TypeError, ap, x, [x[0], x[1].half()], cache, tb, ln)                # types
    bad(TypeError, ap, [t.float() for t in x], x, cache, tb, ln)
    bad(ValueError, ap, [t[:, :1] for t in x], x, cache, tb, ln)             # heads
    bad(ValueError, ap, x, [x[0], x[1].transpose(1, 2).contiguous().transpose(1, 2)], cache, tb, ln)     # strides
    bad(ValueError, ap, x, x, cache, tb, ln[:2])
    bad(ValueError, ap, x, x, cache, tb.long(), ln)
    bad(ValueError, ap, x, x, cache, tb, ln, cu_new=torch.zeros(3, dtype=torch.int32, device=DEV))
    bad(ValueError, ap, x, x, cache, tb, ln, cos)                            # cos without sin
    bad(TypeError, ap, x, x, cache, tb, ln, cos.half(), cos.half())
    bad(coc.CocError, ap, x, x, cache, tb, ln, torch.zeros(4, 40, device=DEV), torch.zeros(4, 40, device=DEV))      # rot_dim > head_dim
    bad(ValueError, ap, x, x, cache, tb, ln, q_outs=q)                       # outputs without qs
    bad(ValueError, ap, x, x, cache, tb, ln, qs=q, q_outs=[q[0], q[1][:, :2]])
    bad(ValueError, at, [t.cpu() for t in q], cache, tb, ln)
    bad(coc.CocError, at, [t[:, :3].contiguous() for t in q], cache, tb, ln)     # 3 query heads on 2
    bad(coc.CocError, at, q, cache, tb, ln, sinks=1)
    bad(coc.CocError, at, q, cache, tb, ln, window=-1)
    bad(TypeError, at, q, object(), tb, ln)
    bad(ValueError, coc.KVCache, cache.k, cache.v[:1], cache.k_scale, cache.v_scale)
    bad(TypeError, coc.KVCache, [t.view(torch.uint8) for t in cache.k], cache.v, cache.k_scale, cache.v_scale)
    f = coc.matmul_all_reduce_w4a16
    xs, ws, sc = [torch.zeros(2, 64, dtype=BF, device=DEV)], [torch.zeros(8, 16, dtype=torch.int32, device=DEV)], [torch.zeros(2, 16, dtype=BF, device=DEV)]
    bad(coc.CocError, f, xs, ws, sc, 48)
    bad(coc.CocError, f, xs, ws, [torch.zeros(4, 16, dtype=BF, device=DEV)], 16)      # groups below 32
    bad(ValueError, f, xs, ws, [sc[0][:1]], 32)
    bad(TypeError, f, xs, ws, [sc[0].half()], 32)
    bad(TypeError, f, xs, [ws[0].long()], sc, 32)
    bad(TypeError, f, xs, ws, sc, 32, zeros=[torch.zeros(2, 16, dtype=torch.int32, device=DEV)])
    bad(coc.CocError, f, xs, [torch.zeros(8, 20, dtype=torch.int32, device=DEV)], [torch.zeros(2, 20, dtype=BF, device=DEV)], 32)   # n % 8
    coc.sync_status()


def guarded(shape, dt):
    """(outputs inside a larger buffer, check that nothing around them changed)."""
    n = 1
    for x in shape:
        n *= x
    buf = torch.full((n + 512,), 7.0, dtype=dt, device=DEV)

    def intact():
        return bool((buf[:256] == 7).all() and (buf[256 + n:] == 7).all())
    return buf[256:256 + n].view(shape), intact


@pytest.mark.parametrize("hq,hkv,d,news,lens", [(5, 1, 80, [3, 1], [90, 7]), (4, 4, 64, [1, 2], [1, 300]), (9, 3, 256, [1], [40])])
def test_nothing_is_written_around_the_outputs(hq, hkv, d, news, lens):
    page = 32
    table, rk, rv, qs = build(1, hq, hkv, d, page, news, lens, BF, seed=31)
    cache = to_cache(rk, rv)
    out, intact = guarded((sum(news), hq, d), BF)
    attend(cache, table, lens, kv.offsets(news), qs, outs=[out])
    coc.sync_status()
    assert intact()
    out, intact = guarded((sum(news), hq, d), BF)
    k = [torch.randn(sum(news), hkv, d, device=DEV).to(BF)]
    cos = torch.ones(max(lens), d // 2, device=DEV)
    coc.kv_cache_append(k, k, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), cos, cos,
                        qs=[q.to(DEV) for q in qs], q_outs=[out], cu_new=torch.tensor(kv.offsets(news), dtype=torch.int32, device=DEV))
    coc.sync_status()
    assert intact()


def test_steady_state_attention_allocates_nothing_and_shutdown_recovers():
    """Repeated calls take their scratch from the stream's workspace, also after it was freed or grew."""
    table, rk, rv, qs = build(1, 8, 1, 128, 64, [1], [5000], BF, seed=12)
    cache, tb = to_cache(rk, rv), table.to(DEV)
    ln = torch.tensor([5000], dtype=torch.int32, device=DEV)
    q = [x.to(DEV) for x in qs]
    want = coc.kv_cache_attention(q, cache, tb, ln)[0].clone()
    torch.cuda.synchronize()
    n = coc.alloc_count()
    for _ in range(5):
        assert torch.equal(coc.kv_cache_attention(q, cache, tb, ln)[0], want)
    assert coc.alloc_count() == n
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [coc.kv_cache_attention(q, cache, tb, ln)[0] for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)
    coc.shutdown()
    assert torch.equal(coc.kv_cache_attention(q, cache, tb, ln)[0], want)
    coc.sync_status()


@pytest.mark.parametrize("dt", [BF, HF])
def test_attention_of_equal_keys_and_of_one_that_dominates(dt):
    """All logits equal: the mean of the values.  One logit far above: its value."""
    g = torch.Generator().manual_seed(14)
    page, d, n = 16, 64, 1000
    table, pages = kv.make_table([n], page, gen=g)
    rv = kv.random_cache(1, pages, 1, page, d, g)
    zero = [(torch.zeros(pages, 1, page, d, dtype=torch.uint8), torch.ones(pages, 1))]
    q = [torch.randn(1, 2, d, generator=g).to(dt)]
    outs = attend(to_cache(zero, rv), table, [n], None, q)
    check(outs, q, zero, rv, table, [n], [0, 1], page)
    one = [(zero[0][0].clone(), zero[0][1])]
    one[0][0][table[0, 30].item(), 0, 5] = 0x78          # 256 in every value of one key
    q = [torch.ones(1, 2, d).to(dt)]
    outs = attend(to_cache(one, rv), table, [n], None, q)
    v = kv.gather(kv.values(*rv[0]), table[0], n, page)[0, 30 * page + 5]
    assert torch.equal(outs[0].cpu()[0], v.to(dt).expand(2, d))


def test_outputs_of_several_ranks_are_ordinary_tensors():
    """New outputs share one allocation: aligned, packed, usable and independent like separate tensors."""
    table, rk, rv, qs = build(3, 4, 2, 80, 32, [1], [40], BF, seed=33)
    outs = attend(to_cache(rk, rv), table, [40], None, qs)
    for o in outs:
        assert o.shape == (1, 4, 80) and o.is_contiguous() and o.data_ptr() % 16 == 0 and not o.requires_grad
    keep = [o.clone() for o in outs]
    outs[1].fill_(3)
    assert torch.equal(outs[0], keep[0]) and torch.equal(outs[2], keep[2]) and (outs[1] == 3).all()
    w = torch.ones(80, device=DEV, dtype=BF, requires_grad=True)
    (outs[2] * w).sum().backward()
    assert w.grad.shape == (80,)
    outs[0].zero_()
    view = outs[0].view(4, 80)[1:]
    assert view.shape == (3, 80) and not view.any()


# Sequences with clearly more than 8 rows behind a table of 4096 tiles or more take tiles of 16 rows.
TALL = [
    # R, hq, hkv, d, page, new tokens, lengths, window, sinks, dtype
    (1, 16, 1, 128, 128, [1, 1], [700, 1], 0, 0, BF),
    (2, 9, 1, 64, 128, [1, 1, 1], [0, 65, 3000], 0, 0, HF),            # one row past a tile of 8, a row that sees nothing
    (1, 20, 1, 80, 64, [2, 0, 3], [500, 50, 2], 0, 0, BF),             # ragged last tile, 3 new tokens of 2 positions
    (1, 8, 2, 128, 32, [6, 1, 4], [300, 64, 4], 0, 0, HF),
    (1, 5, 1, 112, 128, [7], [1029], 100, 4, BF),                      # rows of one tile with different windows
    (2, 24, 2, 128, 64, [3, 2], [300, 2000], 1, 0, BF),
    (1, 4, 4, 48, 16, [19, 5], [210, 17], 33, 70, HF),
    (1, 32, 2, 16, 128, [1], [20000], 0, 0, BF),                       # split over many blocks
]


@pytest.mark.parametrize("R,hq,hkv,d,page,news,lens,window,sinks,dt", TALL)
def test_attention_tiles_of_16_rows(R, hq, hkv, d, page, news, lens, window, sinks, dt):
    table, rk, rv, qs = build(R, hq, hkv, d, page, news, lens, dt, seed=d + page, width=4096 * 64 // page)
    cache, cu = to_cache(rk, rv), kv.offsets(news)
    outs = attend(cache, table, lens, cu, qs, window=window, sinks=sinks)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, cu, page, window, sinks)
    again = attend(cache, table, lens, cu, qs, window=window, sinks=sinks)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("d,hq", [(128, 12), (64, 5)])
def test_attention_tiles_of_16_rows_nan(d, hq):
    """As with tiles of 8 rows: a NaN value reaches only the rows that see it, in its place, a NaN key only the rows that see it."""
    news, lens = [3], [50]
    table, rk, rv, qs = build(1, hq, 1, d, 16, news, lens, BF, seed=6, width=16384)
    page48 = table[0, 3].item()
    ref, size, reach = kv.attention(qs[0], kv.values(*rk[0]), kv.values(*rv[0]), table, lens, [0, 3], 16, d ** -0.5)
    bound = kv.attention_bound(ref, size, reach, 50, BF)
    bad_v, bad_k = rv[0][0].clone(), rk[0][0].clone()
    bad_v[page48, 0, 0, 7] = kv.NAN_CODE         # position 48: seen by new tokens 1 and 2
    bad_k[page48, 0, 1, 3] = kv.NAN_CODE         # position 49: seen by new token 2 alone
    got = attend(to_cache(rk, [(bad_v, rv[0][1])]), table, lens, [0, 3], qs)[0].cpu().double()
    assert torch.isnan(got[1:, :, 7]).all()
    rest = [i for i in range(d) if i != 7]
    assert ((got - ref).abs() <= bound)[:, :, rest].all()
    assert ((got - ref).abs() <= bound)[0].all()
    got = attend(to_cache([(bad_k, rk[0][1])], rv), table, lens, [0, 3], qs)[0].cpu().double()
    assert torch.isnan(got[2]).all()
    assert ((got - ref).abs() <= bound)[:2].all()
    coc.sync_status()


@pytest.mark.parametrize("seed,q_std,k_exp,v_exp", [(1, 30.0, 0, 0), (3, 1.0, -40, 30), (4, 1.0, 0, -60), (5, 6e4, -20, 0)])
def test_attention_tiles_of_16_rows_ranges(seed, q_std, k_exp, v_exp):
    news, lens = [1, 2], [150, 333]
    table, rk, rv, qs = build(1, 24, 2, 128, 32, news, lens, BF, seed, q_std=q_std, width=8192)
    rk = [(c, s * 2.0 ** k_exp) for c, s in rk]
    rv = [(c, s * 2.0 ** v_exp) for c, s in rv]
    scale = 128 ** -0.5 * 2.0 ** -k_exp / (q_std if q_std > 100 else 1.0)
    outs = attend(to_cache(rk, rv), table, lens, kv.offsets(news), qs, scale=scale)
    coc.sync_status()
    check(outs, qs, rk, rv, table, lens, kv.offsets(news), 32, scale=scale)
