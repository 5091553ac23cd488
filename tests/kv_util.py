"""Plain 64-bit definitions of the paged 8-bit key/value cache's operators, and
random caches for their tests.  Everything here is CPU torch in float64."""
import torch

E4M3 = torch.float8_e4m3fn
NAN_CODE = 0x7F


def e4m3(x):
    """The nearest e4m3 value of each float64 value: ties to even, saturating."""
    mag = x.abs().clamp(max=448.0)
    _, e = torch.frexp(mag)
    ulp = torch.ldexp(torch.ones_like(mag), (e - 1).clamp(min=-6) - 3)
    return torch.sign(x) * torch.minimum(torch.round(mag / ulp) * ulp, torch.full_like(mag, 448.0))


def page_scale(amax: float) -> float:
    """The least power of two s >= 2**-100 with amax <= 448 s."""
    s = 2.0 ** -100
    while amax > 448.0 * s:
        s *= 2.0
    return s


def offsets(news):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return cu


def make_table(lens, page, width=None, spare=2, gen=None):
    """(block table with -1 where nothing is stored, pages): shuffled pages."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    width = max(1, max(need, default=0)) if width is None else width
    perm = torch.randperm(pages, generator=gen).tolist()
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        for i in range(min(n, width)):
            t[s, i] = perm.pop()
    return t, pages


def random_cache(R, pages, heads, page, d, gen, spread=0.5):
    """[(codes as uint8, scales)] per rank: normal values, a scale of its own for every page and head."""
    out = []
    for _ in range(R):
        x = torch.randn(pages, heads, page, d, generator=gen, dtype=torch.float64)
        x = x * torch.exp(spread * torch.randn(pages, heads, 1, 1, generator=gen, dtype=torch.float64))
        top = x.abs().amax((2, 3)).reshape(-1).tolist()
        s = torch.tensor([page_scale(v) for v in top], dtype=torch.float64).view(pages, heads)
        out.append((e4m3(x / s[:, :, None, None]).to(torch.float32).to(E4M3).view(torch.uint8), s.float()))
    return out


def values(u8, scale):
    return u8.view(E4M3).to(torch.float64) * scale.double()[:, :, None, None]


def gather(vals, table_row, n, page):
    """(heads, n, d) of one sequence's first n positions."""
    ids = table_row[: -(-n // page)].long()
    return vals[ids].transpose(0, 1).reshape(vals.shape[1], -1, vals.shape[3])[:, :n]


def visible(end, window, sinks):
    """Positions a row whose keys end at `end` sees."""
    if end <= 0:
        return []
    a = max(0, end - window) if window else 0
    return list(range(min(a, sinks))) + list(range(a, end))


def attention(q, kv, vv, table, lens, cu, page, scale, window=0, sinks=0):
    """(out, weight of |v|, largest sum of |q k|) in float64: out[t, h], sum_j p_j |v_j| and max_j scale sum_d |q_d k_jd|."""
    T, hq, d = q.shape
    H = kv.shape[1]
    G = hq // H
    out, size, reach = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, 1, dtype=torch.float64)
    for s, n in enumerate(lens):
        if n <= 0 or cu[s + 1] == cu[s]:
            continue
        k, v = gather(kv, table[s], n, page), gather(vv, table[s], n, page)
        for t in range(cu[s], cu[s + 1]):
            seen = visible(n - (cu[s + 1] - 1 - t), window, sinks)
            if not seen:
                continue
            x = q[t].double().view(H, G, d)
            z = x @ k[:, seen].transpose(1, 2) * scale
            p = torch.softmax(z, 2)
            out[t] = (p @ v[:, seen]).view(hq, d)
            size[t] = (p @ v[:, seen].abs()).view(hq, d)
            reach[t] = ((x.abs() @ k[:, seen].abs().transpose(1, 2)) * scale).amax(2).view(hq, 1)
    return out, size, reach


def unit(dtype):
    """Unit roundoff of a 16-bit type."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11


def attention_bound(ref, size, reach, keys, dtype):
    """The output's rounding; weights held in 11 bits or more (2**-11 of sum p |v|); logits summed in fp32 over at most 256
    products (2**-15 of their size, in numerator and denominator); sums over the keys at 2**-23 a step; the least fp16."""
    return unit(dtype) * ref.abs() + (2.0 ** -11 + 2.0 ** -15 * reach + keys * 2.0 ** -23) * size + 2.0 ** -24
