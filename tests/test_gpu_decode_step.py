"""The attention block of a decode step (QKV projection, append, attention over
the 8-bit cache, w4A16 output projection) against a float64 composition whose
cache is the one the step left."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc
from tensor_matmul_collective_gb300 import decode_step as ds

import kv_util as kv
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def reference(block, xs, table, lens, cu, page):
    """Output in float64 from the block's inputs and what its cache holds now."""
    hq, hk, d = block.q_heads, block.kv_heads, block.head_dim
    x = torch.cat([t.double().cpu() for t in xs])
    cos, sin = block.cos.double().cpu(), block.sin.double().cpu()
    pos = torch.cat([torch.arange(n - (cu[s + 1] - cu[s]), n) for s, n in enumerate(lens)])
    y = 0.0
    for r in range(len(xs)):
        q = (x @ block.w_qkv[r].double().cpu())[:, :hq * d].view(-1, hq, d)
        a, b = q[..., :d // 2], q[..., d // 2:]
        c, s = cos[pos][:, None], sin[pos][:, None]
        q = torch.cat((a * c - b * s, b * c + a * s), -1)
        k = kv.values(block.cache.k[r].view(torch.uint8).cpu(), block.cache.k_scale[r].cpu())
        v = kv.values(block.cache.v[r].view(torch.uint8).cpu(), block.cache.v_scale[r].cpu())
        out, _, _ = kv.attention(q, k, v, table, lens, cu, page, d ** -0.5, block.window, block.sinks)
        words = block.w_out[r].cpu().long()
        codes = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], 1).reshape(-1, words.shape[1]).double()
        w = (codes - 8.0) * block.scales[r].double().cpu().repeat_interleave(block.group, 0)
        y = y + out.reshape(out.shape[0], hq * d) @ w
    return y


@pytest.mark.parametrize("R,heads,kv_heads,dtype,window", [(2, 8, 4, torch.bfloat16, 0), (1, 4, 1, torch.float16, 40), (4, 8, 4, torch.bfloat16, 0)])
def test_prompts_then_single_tokens(R, heads, kv_heads, dtype, window):
    hidden, d, page = 256, 64, 32
    block = ds.random_block(R, hidden, heads, kv_heads, d, pages=40, page_size=page, positions=300, dtype=dtype, seed=R,
                            window=window, sinks=4 if window else 0)
    g = torch.Generator().manual_seed(R)
    B = 8 * R
    news = [3 if s % 2 else 5 for s in range(B)]
    news[0] += 8 * R * (-(-sum(news) // (8 * R))) - sum(news)      # a whole number of 8-row shards
    lens = list(news)
    need = [-(-(n + 3) // page) for n in lens]
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    perm = torch.randperm(40, generator=g).tolist()
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = perm.pop()
    cu = kv.offsets(news)
    for step in range(3):
        tokens = cu[-1]
        xs = [torch.randn(tokens // R, hidden, generator=g).to(dtype).to(DEV) for _ in range(R)]
        outs = block(xs, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                     cu_new=None if step else torch.tensor(cu, dtype=torch.int32, device=DEV))
        coc.sync_status()
        ref = reference(block, xs, table, lens, cu, page)
        err = outs[0].double().cpu() - ref
        # q, its rotation and the context are rounded to 16 bits on the way, each a relative 2**-9 at most (bf16), and logits of
        # size up to about 4 carry q's error into the weights; independent errors: a few thousandths of the result's norm
        unit = kv.unit(dtype)
        assert float(err.norm() / ref.norm()) <= 4 * unit
        assert all(torch.equal(o, outs[0]) for o in outs)
        lens = [n + 1 for n in lens]
        cu = list(range(B + 1))
