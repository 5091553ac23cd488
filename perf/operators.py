"""The decode-step operators of a tensor-parallel attention block, as cases that can be timed and compared.

Three operators, every one over R rank shards in one call:

* append: rotate q and k by position and append k and v to a paged cache held in 8 bits (e4m3 codes, one
  power-of-two scale for each page and key/value head),
* attend: attention of a few new tokens per sequence over that cache, optionally with a sliding window and a
  few first tokens that stay visible,
* w4: the row-parallel product with 4-bit weights and group scales, summed over the ranks.

``run`` computes them in elementary torch operations in 32 bits, or (``own``) through the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
MIN_EXP = -100          # the least scale of a page is 2**MIN_EXP


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # --- append: bytes are the new tokens' q, k, v and the codes written
        # one user's next token on one rank: only the launch counts
        {"name": "append_one_token", "op": "append", "R": 1, "seqs": 1, "new": 1, "past": 777, "hq": 8,
         "hkv": 1, "d": 128, "rot": 128, "page": 64, "interleaved": False, "dtype": "bf16"},
        # a serving batch's next tokens, 8 ranks of a layer with 64 query and 8 key/value heads
        {"name": "append_decode_batch", "op": "append", "R": 8, "seqs": 128, "new": 1, "past": 160,
         "hq": 8, "hkv": 1, "d": 128, "rot": 128, "page": 64, "interleaved": False, "dtype": "bf16"},
        # prompts of unlike lengths, some of them continued in the middle of a page
        {"name": "append_prompts", "op": "append", "R": 8, "seqs": 7, "new": 2047, "past": 300, "hq": 8,
         "hkv": 1, "d": 128, "rot": 128, "page": 64, "interleaved": False, "dtype": "bf16"},
        # --- attend: bytes are the visible keys and values
        # one user, a short context, all heads on one rank
        {"name": "attend_one_short", "op": "attend", "R": 1, "seqs": 1, "new": 1, "low": 777, "high": 777, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a serving batch of unlike lengths, 8 ranks of a layer with 64 query and 8 key/value heads
        {"name": "attend_decode_batch", "op": "attend", "R": 8, "seqs": 48, "new": 1, "low": 1, "high": 8192, "hq": 8,
         "hkv": 1, "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # two users with very long contexts
        {"name": "attend_two_long", "op": "attend", "R": 8, "seqs": 2, "new": 1, "low": 130000, "high": 131071, "hq": 8,
         "hkv": 1, "d": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # drafted tokens being verified, one query head for each key/value head (32 heads over 8 ranks), small pages
        {"name": "attend_verify_mha", "op": "attend", "R": 8, "seqs": 16, "new": 5, "low": 3, "high": 2048, "hq": 4,
         "hkv": 4, "d": 128, "page": 16, "window": 0, "sinks": 0, "dtype": "fp16"},
        # a sliding window with sink tokens over longer contexts, 80 values a head
        {"name": "attend_window_sinks", "op": "attend", "R": 4, "seqs": 33, "new": 2, "low": 1000, "high": 6000, "hq": 8,
         "hkv": 2, "d": 80, "page": 32, "window": 1023, "sinks": 4, "dtype": "bf16"},
        # --- w4: bytes are the 4-bit weights
        # one token through a square layer of one rank
        {"name": "w4_one_token", "op": "w4", "R": 1, "m": 1, "n": 4096, "ks": 4096, "group": 128, "zeros": False,
         "dtype": "bf16"},
        # the output projection behind the attention above: 8 ranks, 8 tokens
        {"name": "w4_out_projection", "op": "w4", "R": 8, "m": 8, "n": 8192, "ks": 1024, "group": 128, "zeros": False,
         "dtype": "bf16"},
        # a layer with 14336 columns at 16 tokens, the largest weight
        {"name": "w4_wide_16", "op": "w4", "R": 8, "m": 16, "n": 14336, "ks": 7168, "group": 128, "zeros": True,
         "dtype": "bf16"},
        # odd sizes: five tokens, ragged columns, small groups with zero points, fp16
        {"name": "w4_odd_fp16", "op": "w4", "R": 2, "m": 5, "n": 8200, "ks": 3584, "group": 32, "zeros": True,
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "w4"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "w4":
        R = rng.choice([1, 2, 4, 8])
        group = rng.choice([32, 64, 128])
        n = 8 * _log(rng, 64, 1792) // 24 * 24 + 8                 # never a multiple of 24
        total = _log(rng, 1 << 20, 8 * 14336 * 7168)               # weights over all ranks
        ks = group * (max(1, min(total // (R * n), 16384) // group) // 3 * 3 + 1)
        return {"op": "w4", "R": R, "m": _log(rng, 1, 16), "n": n, "ks": ks, "group": group,
                "zeros": rng.random() < 0.5, "dtype": dtype}
    R = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 80, 96, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8]) if R <= 2 else rng.choice([1, 2])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        prompts = rng.random() < 0.5
        tokens = _log(rng, 1, 4096)
        tokens = max(1, min(tokens, (8192 * 8 * 10 * 128) // (R * (hq + 2 * hkv) * d)))
        if prompts:
            seqs = rng.randint(1, 8)
            new = max(2, tokens // seqs)
        else:
            seqs, new = max(1, min(tokens, 256)), 1
        return {"op": "append", "R": R, "seqs": seqs, "new": new, "past": rng.randint(0, 300),
                "hq": hq, "hkv": hkv, "d": d, "rot": d if rng.random() < 0.7 else d // 2, "page": page,
                "interleaved": rng.random() < 0.3, "dtype": dtype}
    high = _log(rng, 16, 131072)
    most = 8 * 2 * 131072 * 128                                    # code pairs of the largest listed case
    seqs = _log(rng, 1, 128)
    seqs = max(1, min(seqs, most // (R * hkv * d * high)))
    high = max(16, min(high, most // (R * hkv * d * seqs)))
    return {"op": "attend", "R": R, "seqs": seqs, "new": rng.choice([1, 1, 1, rng.randint(2, 8)]),
            "low": rng.choice([1, high // 2, high]), "high": high, "hq": hq, "hkv": hkv, "d": d, "page": page,
            **rng.choice([{"window": 0, "sinks": 0}, {"window": 0, "sinks": 0},
                          {"window": _log(rng, 16, 4096), "sinks": rng.choice([0, 1, 4, 100])}]), "dtype": dtype}


# ----------------------------------------------------------------- inputs ---

def _lengths(case, seed):
    """(new tokens, tokens in the cache with them) of each sequence, as lists. The new tokens' counts are the case's, in an
    order that goes by the seed, so that every seed's outputs have the same shapes."""
    r = random.Random(len(str(sorted(case.items()))) * 7907 + case["seqs"] * 31 + case["new"])
    B, new = case["seqs"], [case["new"]] * case["seqs"]
    if case["new"] > 1:
        new[1:] = [r.randint(0 if case["op"] == "append" else 1, case["new"]) for _ in range(B - 1)]
    r = random.Random(1000003 * seed + 17)
    r.shuffle(new)
    if case["op"] == "append":
        return new, [n + r.randint(0, case["past"]) for n in new]
    lens = [r.randint(case["low"], case["high"]) for _ in range(B)]
    lens[r.randrange(B)] = case["high"]
    return new, lens


def _pool(case, new):
    """Pages of a cache that holds the longest sequences of the case, and one that none uses."""
    most = [n + case["past"] for n in new] if case["op"] == "append" else [case["high"]] * case["seqs"]
    return sum(-(-n // case["page"]) for n in most) + 1


def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s (448 is the largest e4m3 value), in float32 by its exponent's bits."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e + torch.where(m > 0.875, -8, -9), torch.full_like(e, MIN_EXP))
    return ((e.clamp(min=MIN_EXP) + 127) << 23).to(torch.int32).view(torch.float32)


def _table(case, lens, pages, g):
    """Block table over a shuffled pool; its unused entries are -1, and no sequence has the last page."""
    need = [-(-n // case["page"]) for n in lens]
    perm = torch.randperm(pages - 1, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(max(1, max(need)), device=DEV)[None, :]
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)[:, None]
    used = at < torch.tensor(need, device=DEV)[:, None]
    return torch.where(used, perm[(first + at).clamp(max=pages - 2)], torch.full_like(perm[:1], -1)).contiguous()


def _cache(case, pages, g, spread):
    """Codes and scales of one rank's keys or values: normal values with a few strong channels, quantised a page at a time."""
    H, page, d = case["hkv"], case["page"], case["d"]
    gain = torch.exp(spread * torch.randn(1, H, 1, d, generator=g, device=DEV))
    codes = torch.empty(pages, H, page, d, dtype=E4M3, device=DEV)
    scale = torch.empty(pages, H, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (H * page * d))
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), H, page, d, generator=g, device=DEV) * gain
        s = _pow2_scale(x.abs().amax((2, 3)))
        scale[a:a + step] = s
        codes[a:a + step] = (x / s[:, :, None, None]).to(E4M3)
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 101)
    dt, R = DTYPES[case["dtype"]], case["R"]
    st = {"case": case}
    if case["op"] == "w4":
        m, n, ks, group = case["m"], case["n"], case["ks"], case["group"]
        st["x"] = [torch.randn(m, ks, generator=g, device=DEV).to(dt) for _ in range(R)]
        # eight 4-bit codes along k in a word: bits 4i..4i+3 of word [t, j] are the code of weight [8 t + i, j]
        st["w"] = [torch.randint(-2 ** 31, 2 ** 31, (ks // 8, n), generator=g, device=DEV, dtype=torch.int32) for _ in range(R)]
        st["scale"] = [(0.001 + 0.009 * torch.rand(ks // group, n, generator=g, device=DEV)).to(dt) for _ in range(R)]
        st["zero"] = [torch.randint(0, 16, (ks // group, n), generator=g, device=DEV, dtype=torch.int8)
                      for _ in range(R)] if case["zeros"] else None
        return st
    H, hq, d = case["hkv"], case["hq"], case["d"]
    new, lens = _lengths(case, seed)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
    single = case["new"] == 1                                     # one new token in every sequence: no offsets are needed
    st["cu"] = None if single else torch.tensor(cu, dtype=torch.int32, device=DEV)
    pages = _pool(case, new)
    st["table"] = _table(case, lens, pages, g)
    made = [(_cache(case, pages, g, 0.7), _cache(case, pages, g, 0.2)) for _ in range(R)]
    st["kv"] = tuple([pair[i][j] for pair in made] for i, j in ((0, 0), (1, 0), (0, 1), (1, 1)))
    if case["op"] == "append":
        # slices of the fused projection's output, as the projection leaves them
        qkv = [torch.randn(T, (hq + 2 * H) * d, generator=g, device=DEV).to(dt) for _ in range(R)]
        st["q"] = [t[:, :hq * d].view(T, hq, d) for t in qkv]
        st["k"] = [t[:, hq * d:(hq + H) * d].view(T, H, d) for t in qkv]
        st["v"] = [t[:, (hq + H) * d:].view(T, H, d) for t in qkv]
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        angle = torch.arange(max(lens), device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    else:
        st["q"] = [(1.5 * torch.randn(T, hq, d, generator=g, device=DEV)).to(dt) for _ in range(R)]
        st["softmax_scale"] = 1.0 / math.sqrt(d)
    if own:
        from tensor_matmul_collective_gb300 import coc
        st["cache"] = coc.KVCache(*st["kv"])
    return st


# -------------------------------------------------------------------- run ---

def run(st):
    op = st["case"]["op"]
    if own:
        from tensor_matmul_collective_gb300 import coc
        if op == "w4":
            return coc.matmul_all_reduce_w4a16(st["x"], st["w"], st["scale"], st["case"]["group"], zeros=st["zero"])
        if op == "attend":
            c = st["case"]
            return coc.kv_cache_attention(st["q"], st["cache"], st["table"], st["lens"], cu_new=st["cu"],
                                          scale=st["softmax_scale"], window=c["window"], sinks=c["sinks"])
        q = coc.kv_cache_append(st["k"], st["v"], st["cache"], st["table"], st["lens"], st["cos"], st["sin"], qs=st["q"],
                                cu_new=st["cu"], interleaved=st["case"]["interleaved"])
        return {"q": q, "cache": st["kv"]}
    if op == "w4":
        return _plain_w4(st)
    return _plain_attend(st) if op == "attend" else _plain_append(st)


def _w4_part(x, w, scale, zero, group):
    ks, n = 8 * w.shape[0], w.shape[1]
    bits = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)[None, :, None]
    code = ((w[:, None, :] >> bits) & 15).float().view(ks // group, group, n)
    z = 8.0 if zero is None else zero.float()[:, None, :]
    return x.float() @ ((code - z) * scale.float()[:, None, :]).view(ks, n)


def _plain_w4(st):
    zero = st["zero"] or [None] * len(st["x"])
    y = sum(_w4_part(x, w, s, z, st["case"]["group"]) for x, w, s, z in zip(st["x"], st["w"], st["scale"], zero))
    y = y.to(st["x"][0].dtype)
    return [y.clone() for _ in st["x"]]


def _tokens(st, T):
    """Sequence and position of every new token, and the number of new tokens of every sequence."""
    B = st["lens"].shape[0]
    cu = torch.arange(B + 1, device=DEV) if st["cu"] is None else st["cu"].long()
    t = torch.arange(T, device=DEV)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    new = cu[1:] - cu[:-1]
    return seq, st["lens"].long()[seq] - new[seq] + t - cu[seq], new


def _rotate(x, cos, sin, interleaved):
    """Rotation of the first 2 * cos.shape[1] values of every head; cos and sin are those of the tokens' positions."""
    half = cos.shape[1]
    x = x.float()
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _scales(x, old, page_of, held):
    """Every page's scale once the values x (arrays, tokens, heads, d) are in it; held: each sequence's page that already
    holds tokens (the unused last page: none)."""
    at = page_of[None, :, None].expand(x.shape[0], -1, x.shape[2])
    amax = torch.zeros_like(old).scatter_reduce_(1, at, x.abs().amax(3), "amax")
    kept = torch.zeros_like(old)
    kept[:, held] = old[:, held]
    touched = torch.zeros(old.shape[1], dtype=torch.bool, device=DEV)
    touched[page_of] = True
    return torch.where(touched[None, :, None], torch.maximum(_pow2_scale(amax), kept), old)


def _store(x, codes, scale, s, page_of, slot, held, keep):
    """New tokens' values x (fp32) into one array's codes, whose scales become s; keep: slots of the held pages with earlier tokens."""
    u8 = codes.view(torch.uint8)
    was = u8[held]
    again = (was.view(E4M3).float() * (scale[held] / s[held])[:, :, None, None]).to(E4M3).view(torch.uint8)
    u8[held] = torch.where(keep[:, None, :, None], again, was)
    u8[page_of, :, slot] = (x / s[page_of][:, :, None]).to(E4M3).view(torch.uint8)
    scale.copy_(s)


def _plain_append(st):
    case = st["case"]
    T, page = st["q"][0].shape[0], case["page"]
    seq, pos, new = _tokens(st, T)
    table = st["table"].long()
    page_of, slot = table[seq, pos // page], pos % page
    past = st["lens"].long() - new
    held = table.gather(1, (past // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    pages = st["kv"][0][0].shape[0]
    held = torch.where((past % page > 0) & (new > 0), held, torch.full_like(held, pages - 1))
    keep = torch.arange(page, device=DEV)[None, :] < (past % page)[:, None]
    cos, sin = st["cos"][pos], st["sin"][pos]
    kc, vc, ks, vs = st["kv"]
    x = torch.cat((_rotate(torch.cat(st["k"]), cos.repeat(len(kc), 1), sin.repeat(len(kc), 1), case["interleaved"]),
                   torch.cat(st["v"]).float())).view(2 * len(kc), T, case["hkv"], case["d"])
    s = _scales(x, torch.stack(ks + vs), page_of, held)
    [_store(*each, page_of, slot, held, keep) for each in zip(x, kc + vc, ks + vs, s)]
    return {"q": [_rotate(q, cos, sin, case["interleaved"]).to(q.dtype) for q in st["q"]], "cache": st["kv"]}


def _attend_rank(q, kc, vc, ks, vs, table, see, rows, scale):
    """One rank. see: (sequences, new, keys) truth values, rows: (sequence, index) of every token."""
    B, W = table.shape
    H, page, d = kc.shape[1:]
    T, hq, _ = q.shape
    M, L = see.shape[1], W * page
    G = hq // H
    at = table.long().clamp(min=0)

    def values(codes, s):
        x = codes.view(torch.uint8)[at].view(E4M3).float() * s[at][..., None, None]      # sequences, pages, heads, slots, d
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, d)

    qp = torch.zeros(B, M, H, G, d, device=DEV)
    qp[rows[0], rows[1]] = q.float().view(T, H, G, d)
    p = qp.permute(0, 2, 1, 3, 4).reshape(B, H, M * G, d) @ values(kc, ks).transpose(2, 3) * scale
    mask = see[:, None, :, None, :].expand(B, 1, M, G, L).reshape(B, 1, M * G, L)
    p = p.masked_fill(~mask, -math.inf)
    top = p.amax(3, keepdim=True)
    p = torch.exp(p - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(3, keepdim=True)
    v = values(vc, vs)
    v = torch.where(see.any(1)[:, None, :, None], v, torch.zeros_like(v))                # nothing that no row sees comes in
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, H, M, G, d).permute(0, 2, 1, 3, 4)[rows[0], rows[1]].reshape(T, hq, d).to(q.dtype)


def _plain_attend(st):
    case = st["case"]
    T = st["q"][0].shape[0]
    seq, pos, new = _tokens(st, T)
    B, M = new.shape[0], case["new"]
    end = (st["lens"].long() - new)[:, None] + torch.arange(M, device=DEV)[None, :] + 1   # keys before this one
    key = torch.arange(st["table"].shape[1] * case["page"], device=DEV)[None, None, :]
    see = key < end[:, :, None]
    if case["window"]:
        see = see & ((key >= end[:, :, None] - case["window"]) | (key < case["sinks"]))
    see = see & (torch.arange(M, device=DEV)[None, :] < new[:, None])[:, :, None]
    rows = (seq, pos - (st["lens"].long() - new)[seq])
    return [_attend_rank(q, kc, vc, ks, vs, st["table"], see, rows, st["softmax_scale"])
            for q, kc, vc, ks, vs in zip(st["q"], *st["kv"])]


# ------------------------------------------------------------------- work ---

def work(case):
    R = case["R"]
    if case["op"] == "w4":
        m, n, ks = case["m"], case["n"], case["ks"]
        groups = ks // case["group"] * n
        return {"bytes": R * (ks * n / 2 + groups * (3 if case["zeros"] else 2) + 2 * m * ks + 2 * m * n),
                "flops": 2.0 * R * m * n * ks}
    hq, H, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    new, lens = _lengths(case, 1)
    T = sum(new)
    if case["op"] == "append":
        values = T * (2 * hq + 2 * H) * d * 2 + T * 2 * H * d       # q twice, k and v once, their codes
        pages = sum(-(-n // page) - (n - k) // page for k, n in zip(new, lens) if k)
        return {"bytes": R * (values + 2 * pages * H * 4) + 4.0 * case["rot"] * T, "flops": 3.0 * R * T * (hq + H) * case["rot"]}
    keys = rows = 0
    for k, n in zip(new, lens):
        lo = max(0, n - k + 1 - case["window"]) if case["window"] else 0
        first = min(lo, case["sinks"])
        keys += n - lo + first
        for i in range(k):
            end = max(0, n - (k - 1 - i))
            a = max(0, end - case["window"]) if case["window"] else 0
            rows += end - a + min(a, case["sinks"])
    return {"bytes": R * H * (keys * 2.0 * d + keys / page * 8) + R * T * hq * d * 4.0, "flops": 4.0 * R * hq * d * rows}


# ------------------------------------------------------------------ exact ---

def _pow2(e):
    """2**e in float64, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest e4m3 value of every float64 value (ties to even), saturating."""
    mag = x.abs().clamp(max=448.0)
    _, e = torch.frexp(mag)
    ulp = _pow2((e - 1).clamp(min=-6) - 3)
    return torch.sign(x) * torch.minimum(torch.round(mag / ulp) * ulp, torch.full_like(mag, 448.0))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "w4":
        return _exact_w4(st)
    return _exact_attend(st) if case["op"] == "attend" else _exact_append(st)


def _exact_w4(st):
    group, y = st["case"]["group"], 0.0
    for r, (x, w, s) in enumerate(zip(st["x"], st["w"], st["scale"])):
        for a in range(0, w.shape[0] * 8, 2048 // group * group):
            t = torch.arange(a, min(a + 2048 // group * group, w.shape[0] * 8), device=DEV)
            code = torch.bitwise_and(torch.bitwise_right_shift(w[t // 8], (4 * (t % 8)).int()[:, None]), 15).double()
            code -= 8.0 if st["zero"] is None else st["zero"][r][t // group].double()
            y = y + torch.matmul(x[:, t].double(), code * s[t // group].double())
    return [y for _ in st["x"]]


def _exact_append(st):
    case = st["case"]
    page, half = case["page"], case["rot"] // 2
    lens = st["lens"].tolist()
    cu = list(range(len(lens) + 1)) if st["cu"] is None else st["cu"].tolist()
    table = st["table"].tolist()

    def turned(x, pos):
        x = x.double()
        out = x.clone()
        i = torch.arange(half, device=DEV)
        ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        c, s = st["cos"][pos].double()[:, None, :], st["sin"][pos].double()[:, None, :]
        out[:, :, ia] = x[:, :, ia] * c - x[:, :, ib] * s
        out[:, :, ib] = x[:, :, ia] * s + x[:, :, ib] * c
        return out

    at = torch.empty(cu[-1], dtype=torch.long, device=DEV)
    for s, n in enumerate(lens):
        at[cu[s]:cu[s + 1]] = torch.arange(n - (cu[s + 1] - cu[s]), n, device=DEV)
    q = [turned(x, at) for x in st["q"]]
    kc, vc, ks, vs = st["kv"]
    codes, scales = [], []
    for src, old_codes, old_scale in ([(turned(x, at), c, s) for x, c, s in zip(st["k"], kc, ks)]
                                      + [(x.double(), c, s) for x, c, s in zip(st["v"], vc, vs)]):
        c, s = old_codes.double(), old_scale.double()
        for b, n in enumerate(lens):
            t, end = cu[b], cu[b + 1]
            while t < end:
                p = n - (end - t)                                   # the position of token t
                j, slot = table[b][p // page], p % page
                count = min(end - t, page - slot)
                x = src[t:t + count]
                top = x.abs().amax((0, 2)) / 448.0
                fit = _pow2(torch.ceil(torch.log2(top.clamp(min=2.0 ** MIN_EXP))))
                if slot:
                    grown = torch.maximum(fit, s[j])
                    c[j, :, :slot] = _round_e4m3(c[j, :, :slot] * (s[j] / grown)[:, None, None])
                    fit = grown
                s[j] = fit
                c[j, :, slot:slot + count] = _round_e4m3(x / fit[None, :, None]).transpose(0, 1)
                t += count
        codes.append(c)
        scales.append(s)
    R = case["R"]
    return {"q": q, "cache": (codes[:R], codes[R:], scales[:R], scales[R:])}


def _exact_attend(st):
    case = st["case"]
    page, H, d, G = case["page"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    lens = st["lens"].tolist()
    cu = list(range(len(lens) + 1)) if st["cu"] is None else st["cu"].tolist()
    outs = []
    for q, kc, vc, ks, vs in zip(st["q"], *st["kv"]):
        o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            ids = st["table"][b, :-(-n // page)].long()
            k = (kc.view(torch.uint8)[ids].view(E4M3).double() * ks[ids].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, d)[:, :n]
            v = (vc.view(torch.uint8)[ids].view(E4M3).double() * vs[ids].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, d)[:, :n]
            for t in range(cu[b], cu[b + 1]):
                end = n - (cu[b + 1] - 1 - t)
                if end <= 0:
                    continue
                a = max(0, end - case["window"]) if case["window"] else 0
                seen = torch.cat((torch.arange(min(a, case["sinks"]), device=DEV), torch.arange(a, end, device=DEV)))
                z = torch.bmm(q[t].double().view(H, G, d), k[:, seen].transpose(1, 2)) * st["softmax_scale"]
                o[t] = torch.bmm(torch.softmax(z, 2), v[:, seen]).view(H * G, d)
        outs.append(o)
    return outs
