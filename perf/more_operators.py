"""The 8-bit feed-forward operators of a tensor-parallel layer, as cases that can be timed and compared.

Four operators, every one over R rank shards in one call. Values in 8 bits are e4m3 codes with power-of-two scales
(e8m0): one for each row and 128 columns of an activation, one for each 128 x 128 block of a weight.

* quantize: an activation's codes and scales,
* norm: residual addition, root-mean-square norm, codes and scales of the result, and the sum,
* matmul: the product of 8-bit activations with 8-bit weights (out x in), summed over the ranks (all_reduce,
  reduce_scatter) or of the gathered rows with every rank's columns (all_gather),
* gated: the gathered rows through the gate's and the up projection's columns, silu(gate) * up, codes and scales.

``run`` computes them in elementary torch operations in 32 bits, or (``own``) through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BLOCK = 128
MIN_EXP = -100          # the least scale is 2**MIN_EXP
EPS = 1e-5


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # --- quantize: bytes are the values read and the codes written
        # attention's output for a decode batch of 64 tokens, 8 query heads of 128 on each of 8 ranks
        {"name": "quantize_decode", "op": "quantize", "R": 8, "rows": 64, "h": 1024, "dtype": "bf16"},
        # the same of a prompt, odd rows, two ranks with 28 heads
        {"name": "quantize_prompt", "op": "quantize", "R": 2, "rows": 4095, "h": 3584, "dtype": "fp16"},
        # --- norm: bytes are x, residual, sum and codes
        # one user's next token on one rank: only the launch counts
        {"name": "norm_one_token", "op": "norm", "R": 1, "rows": 1, "h": 4096, "residual": True, "dtype": "bf16"},
        # the rows of a prompt of 8192 tokens, sequence parallel over 8 ranks
        {"name": "norm_prompt", "op": "norm", "R": 8, "rows": 1024, "h": 8192, "residual": True, "dtype": "bf16"},
        # first norm of a model (no residual yet), rows whose last block of 128 is cut short, fp16
        {"name": "norm_ragged_fp16", "op": "norm", "R": 2, "rows": 777, "h": 5008, "residual": False, "dtype": "fp16"},
        # --- matmul: operations of the product; for few rows the weights' bytes
        # one token through a square layer of one rank
        {"name": "matmul_one_token", "op": "matmul", "kind": "all_reduce", "R": 1, "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # the down projection of a decode batch, 8 ranks
        {"name": "matmul_down_decode", "op": "matmul", "kind": "all_reduce", "R": 8, "m": 64, "n": 8192, "k": 3584, "dtype": "bf16"},
        # the same layer of a prompt of 4096 tokens, sequence parallel: the largest product
        {"name": "matmul_down_prompt", "op": "matmul", "kind": "reduce_scatter", "R": 8, "m": 4096, "n": 8192, "k": 3584, "dtype": "bf16"},
        # a column-parallel projection with odd rows, columns and inner size, fp16
        {"name": "matmul_ragged_fp16", "op": "matmul", "kind": "all_gather", "R": 2, "m": 333, "n": 1384, "k": 4112, "dtype": "fp16"},
        # --- gated: operations of the two products; for few rows the weights' bytes
        # one token on one rank, a feed-forward size that is no multiple of 128 for every rank count (11008 = 8 x 1376)
        {"name": "gated_one_token", "op": "gated", "R": 1, "m": 1, "f": 11008, "k": 4096},
        # a decode batch of 64 tokens, sequence parallel over 8 ranks
        {"name": "gated_decode", "op": "gated", "R": 8, "m": 8, "f": 3584, "k": 8192},
        # a prompt of 4096 tokens, the largest case
        {"name": "gated_prompt", "op": "gated", "R": 8, "m": 512, "f": 3584, "k": 8192},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "matmul", "matmul", "gated"])
    R = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("quantize", "norm"):
        h = 16 * _log(rng, 8, 1024)
        rows = max(1, min(_log(rng, 1, 8192), (8 * 1024 * 8192) // (R * h)))
        case = {"op": op, "R": R, "rows": rows, "h": h, "dtype": dtype}
        return {**case, "residual": rng.random() < 0.7} if op == "norm" else case
    k = 16 * _log(rng, 16, 512)
    if op == "gated":
        f, m = 16 * _log(rng, 8, 512), _log(rng, 1, 1024)
        m = max(1, min(m, 4096 * 28672 * 8192 // (R * R * f * k)))
        return {"op": op, "R": R, "m": m, "f": f, "k": k}
    kind = rng.choice(["all_reduce", "reduce_scatter", "all_gather"])
    n, m = 8 * _log(rng, 16, 1792), _log(rng, 1, 4096)
    if kind == "all_gather":
        n, m = max(128, n // R // 8 * 8), max(1, m // R)
    if kind == "reduce_scatter":
        m = max(1, m // R) * R
    return {"op": op, "kind": kind, "R": R, "m": m, "n": n, "k": k, "dtype": dtype}


# ----------------------------------------------------------------- inputs ---

def _ceil(a, b=BLOCK):
    return -(-a // b)


def _scale_bits(amax):
    """Exponent + 127 of the least power of two s with amax <= 448 s (448 is the largest e4m3 value), by frexp."""
    mant, e = torch.frexp(amax)
    e = torch.where(amax > 0, e + torch.where(mant > 0.875, -8, -9), torch.full_like(e, MIN_EXP))
    return (e.clamp(min=MIN_EXP) + 127).to(torch.uint8)


def _value(scale):
    """float32 values of e8m0 scales."""
    return (scale.view(torch.uint8).to(torch.int32) << 23).view(torch.float32)


def _spread(scale, h):
    """A row's scales (rows, blocks), for its h columns."""
    return _value(scale).repeat_interleave(BLOCK, 1)[:, :h]


def _codes(y):
    """Codes and scales of float32 rows, a scale for each row and 128 columns."""
    rows, h = y.shape
    blocks = torch.nn.functional.pad(y, (0, _ceil(h) * BLOCK - h)).view(rows, _ceil(h), BLOCK)
    s = _scale_bits(blocks.abs().amax(2)).view(E8M0)
    return (y / _spread(s, h)).to(E4M3), s


def _activation(g, rows, h, gain):
    return torch.randn(rows, h, generator=g, device=DEV) * gain


def _weight(g, n, k):
    """Codes and 128 x 128 scales of an n x k weight with rows of unlike strength."""
    w = torch.randn(n, k, generator=g, device=DEV) * (torch.exp(0.4 * torch.randn(n, 1, generator=g, device=DEV)) * k ** -0.5)
    nb, kb = _ceil(n), _ceil(k)
    t = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
    s = _scale_bits(t.abs().amax((1, 3))).view(E8M0)
    v = _value(s)
    return (t / v[:, None, :, None]).to(E4M3).view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 211)
    R, st = case["R"], {"case": case}
    if case["op"] in ("quantize", "norm"):
        dt, rows, h = DTYPES[case["dtype"]], case["rows"], case["h"]
        # a few strong channels, as hidden states have
        gain = torch.exp(0.7 * torch.randn(1, h, generator=g, device=DEV))
        st["x"] = [_activation(g, rows, h, gain).to(dt) for _ in range(R)]
        if case["op"] == "norm":
            st["weight"] = (1.0 + 0.2 * torch.randn(h, generator=g, device=DEV)).to(dt)
            st["residual"] = [_activation(g, rows, h, gain).to(dt) for _ in range(R)] if case["residual"] else None
        return st
    m, k = case["m"], case["k"]
    gain = torch.exp(0.5 * torch.randn(1, k, generator=g, device=DEV))
    # the ranks' activations as the operators before leave them: parts of one allocation
    x, xs = _codes(_activation(g, R * m, k, gain))
    st["x"], st["xs"] = list(x.view(R, m, k).unbind(0)), list(xs.view(R, m, _ceil(k)).unbind(0))
    if case["op"] == "matmul":
        made = [_weight(g, case["n"], k) for _ in range(R)]
    else:
        halves = [(_weight(g, case["f"], k), _weight(g, case["f"], k)) for _ in range(R)]
        made = [(torch.cat((a[0].view(torch.uint8), b[0].view(torch.uint8))).view(E4M3),
                 torch.cat((a[1].view(torch.uint8), b[1].view(torch.uint8))).view(E8M0)) for a, b in halves]
    st["w"], st["ws"] = [a for a, _ in made], [b for _, b in made]
    return st


# -------------------------------------------------------------------- run ---

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from tensor_matmul_collective_gb300 import coc
        if op == "quantize":
            codes, scales = coc.quantize_f8(st["x"])
            return {"codes": codes, "scales": scales}
        if op == "norm":
            codes, scales, sums = coc.add_rms_norm_f8(st["x"], st["weight"], residuals=st["residual"], eps=EPS)
            return {"codes": codes, "scales": scales, "sums": sums}
        if op == "gated":
            codes, scales = coc.all_gather_gated_matmul_f8(st["x"], st["xs"], st["w"], st["ws"])
            return {"codes": codes, "scales": scales}
        call = {"all_reduce": coc.matmul_all_reduce_f8, "reduce_scatter": coc.matmul_reduce_scatter_f8,
                "all_gather": coc.all_gather_matmul_f8}[case["kind"]]
        return call(st["x"], st["xs"], st["w"], st["ws"], dtype=DTYPES[case["dtype"]])
    return {"quantize": _plain_quantize, "norm": _plain_norm, "matmul": _plain_matmul, "gated": _plain_gated}[op](st)


def _split(ts, R):
    return list(ts.view(R, ts.shape[0] // R, ts.shape[1]).unbind(0))


def _plain_quantize(st):
    codes, scales = _codes(torch.cat(st["x"]).float())
    R = len(st["x"])
    return {"codes": _split(codes, R), "scales": _split(scales, R)}


def _plain_norm(st):
    R = len(st["x"])
    s = torch.cat(st["x"]).float()
    sums = None
    if st["residual"] is not None:
        s = s + torch.cat(st["residual"]).float()
        sums = _split(s.to(st["weight"].dtype), R)
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * st["weight"].float()
    codes, scales = _codes(y)
    return {"codes": _split(codes, R), "scales": _split(scales, R), "sums": sums}


def _real(codes, scale):
    """float32 values of an activation."""
    return codes.float() * _spread(scale, codes.shape[1])


def _real_weight(codes, scale):
    """float32 values of a weight."""
    n, k = codes.shape
    return codes.float() * _spread(scale, k).repeat_interleave(BLOCK, 0)[:n]


def _plain_matmul(st):
    case = st["case"]
    dt, R = DTYPES[case["dtype"]], case["R"]
    if case["kind"] == "all_gather":
        x = torch.cat([_real(c, s) for c, s in zip(st["x"], st["xs"])])
        return [(x @ _real_weight(w, s).t()).to(dt) for w, s in zip(st["w"], st["ws"])]
    y = sum(_real(c, cs) @ _real_weight(w, ws).t() for c, cs, w, ws in zip(st["x"], st["xs"], st["w"], st["ws"])).to(dt)
    return [y.clone() for _ in range(R)] if case["kind"] == "all_reduce" else [t.clone() for t in y.chunk(R)]


def _plain_gated(st):
    f = st["case"]["f"]
    fb = _ceil(f)
    x = torch.cat([_real(c, s) for c, s in zip(st["x"], st["xs"])])
    made = []
    for w, s in zip(st["w"], st["ws"]):
        gate = x @ _real_weight(w[:f], s[:fb]).t()
        up = x @ _real_weight(w[f:], s[fb:]).t()
        made.append(_codes(gate / (1.0 + torch.exp(-gate)) * up))
    return {"codes": [c for c, _ in made], "scales": [s for _, s in made]}


# ------------------------------------------------------------------- work ---

def work(case):
    R = case["R"]
    if case["op"] in ("quantize", "norm"):
        values = R * case["rows"] * case["h"]
        each, flops = 3.0, 3.0
        if case["op"] == "norm":
            each, flops = (7.0 if case["residual"] else 3.0), 7.0
        return {"bytes": values * each + R * case["rows"] * _ceil(case["h"]) + 2.0 * case["h"] * (case["op"] == "norm"),
                "flops": flops * values}
    m, k = case["m"], case["k"]
    read = R * m * (k + _ceil(k))
    if case["op"] == "gated":
        f = case["f"]
        return {"bytes": read + 2.0 * R * (f * k + _ceil(f) * _ceil(k)) + R * R * m * (f + _ceil(f)), "flops": 4.0 * R * R * m * f * k}
    n = case["n"]
    read += R * (n * k + _ceil(n) * _ceil(k))
    if case["kind"] == "all_gather":
        return {"bytes": read + 2.0 * R * R * m * n, "flops": 2.0 * R * R * m * n * k}
    return {"bytes": read + 2.0 * m * n * (R if case["kind"] == "all_reduce" else 1), "flops": 2.0 * R * m * n * k}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    """In 64 bits. A code stands for y / S, which is given unrounded, like every other result here; the scales themselves are
    steps (a power of two or the next), not near a value, and are left out."""
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return {"codes": [_exact_quotient(x.double()) for x in st["x"]], "scales": None}
    if case["op"] == "norm":
        codes, sums = [], []
        for r, x in enumerate(st["x"]):
            s = x.double() if st["residual"] is None else x.double() + st["residual"][r].double()
            norm = torch.sqrt(torch.einsum("ij,ij->i", s, s) / case["h"] + EPS)
            codes.append(_exact_quotient(s / norm[:, None] * st["weight"].double()))
            sums.append(s)
        return {"codes": codes, "scales": None, "sums": None if st["residual"] is None else sums}
    if case["op"] == "gated":
        f, codes = case["f"], []
        for w, s in zip(st["w"], st["ws"]):
            gate = _exact_product(st["x"], st["xs"], w[:f], s[:_ceil(f)])
            gate = gate * torch.sigmoid(gate)
            gate *= _exact_product(st["x"], st["xs"], w[f:], s[_ceil(f):])
            codes.append(_exact_quotient(gate))
        return {"codes": codes, "scales": None}
    if case["kind"] == "all_gather":
        return [_exact_product(st["x"], st["xs"], w, s) for w, s in zip(st["w"], st["ws"])]
    y = 0.0
    for x, xs, w, ws in zip(st["x"], st["xs"], st["w"], st["ws"]):
        y = y + _exact_product([x], [xs], w, ws)
    rows = case["m"] // case["R"]
    return [y] * case["R"] if case["kind"] == "all_reduce" else [y[r * rows:(r + 1) * rows] for r in range(case["R"])]


def _exact_quotient(y):
    """y over its block's scale, block by block."""
    out = torch.empty_like(y)
    for a in range(0, y.shape[1], BLOCK):
        top = y[:, a:a + BLOCK].abs().amax(1)
        frac, e = torch.frexp((top / 448.0).clamp(min=2.0 ** MIN_EXP))
        out[:, a:a + BLOCK] = torch.ldexp(y[:, a:a + BLOCK], torch.where(frac > 0.5, -e, 1 - e)[:, None])
    return out


def _exact_product(xs, x_scales, w, w_scale):
    """Rows of all xs with w, added up block by block of the inner dimension."""
    k = w.shape[1]
    y = torch.zeros(sum(x.shape[0] for x in xs), w.shape[0], dtype=torch.float64, device=DEV)
    row_block = torch.arange(w.shape[0], device=DEV) // BLOCK
    for a in range(0, k, 8 * BLOCK):
        col = torch.arange(a, min(k, a + 8 * BLOCK), device=DEV) // BLOCK
        wd = w[:, a:a + 8 * BLOCK].double() * w_scale.double()[row_block][:, col]
        xd = torch.cat([x[:, a:a + 8 * BLOCK].double() * s.double()[:, col] for x, s in zip(xs, x_scales)])
        y.addmm_(xd, wd.t())
    return y
