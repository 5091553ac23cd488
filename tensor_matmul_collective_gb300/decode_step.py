"""The blocks of a decode step over R tensor-parallel ranks, from the
operators of ``coc``.  Attention: the fused QKV projection (ALL_GATHER_MATMUL of
the sequence-parallel input), append to the 8-bit key/value cache with the
position rotation, attention over the cache, and the output projection with
4-bit weights (w4A16 MATMUL_ALL_REDUCE).  Feed-forward, in 8-bit floating point:
residual addition and RMS norm, gate and up projection with the activation
(ALL_GATHER), down projection (MATMUL_REDUCE_SCATTER).

``python -m tensor_matmul_collective_gb300.decode_step`` appends the keys and
values of prompts to the cache (their own attention is not part of it) and then
runs a number of single-token steps of one layer with random weights and prints
the time of a step (``--ranks 8 --hidden 8192 --heads 64 --kv-heads 8 --batch 64``
by default; the step is captured into a CUDA graph).  With ``--ffn 28672`` the
feed-forward block of that size follows the attention block in every step.
"""
from __future__ import annotations

import argparse

import torch

from . import coc


class AttentionBlock:
    """One layer's attention on R ranks: rank r holds heads/R query heads and
    kv_heads/R key/value heads.

    w_qkv[r]: hidden x (q_heads + 2 kv_heads) head_dim (q, then k, then v), in
    the activations' type.  w_out[r]: (q_heads head_dim / 8) x hidden words of
    4-bit codes (coc.w4_pack) with scales[r] and optional zeros[r] per group."""

    def __init__(self, w_qkv, w_out, scales, group: int, q_heads: int, kv_heads: int, head_dim: int, cos, sin, cache, zeros=None,
                 window: int = 0, sinks: int = 0):
        self.w_qkv, self.w_out, self.scales, self.zeros, self.group = w_qkv, w_out, scales, zeros, group
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.cos, self.sin, self.cache = cos, sin, cache
        self.window, self.sinks = window, sinks

    def __call__(self, xs, block_table, lens, cu_new=None, outs=None, stream=None):
        """xs[r]: rank r's rows of the new tokens' activations (tokens/R x
        hidden, tokens/R a multiple of 8); lens, block_table, cu_new as in
        coc.kv_cache_append.  Returns tokens x hidden on every rank.  With a
        stream everything that is allocated on the way is that stream's."""
        if stream is not None and coc._stream(stream) != torch.cuda.current_stream().cuda_stream:
            now = torch.cuda.current_stream()
            with torch.cuda.stream(coc._as_stream(stream)):
                new = self(xs, block_table, lens, cu_new=cu_new, outs=outs)
            if outs is None:
                new[0].record_stream(now)       # all ranks' are one allocation
            return new
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        qkv = coc.all_gather_matmul(xs, self.w_qkv)
        tokens = qkv[0].shape[0]
        q = [t[:, :hq * d].view(tokens, hq, d) for t in qkv]
        k = [t[:, hq * d:(hq + hk) * d].view(tokens, hk, d) for t in qkv]
        v = [t[:, (hq + hk) * d:].view(tokens, hk, d) for t in qkv]
        q = coc.kv_cache_append(k, v, self.cache, block_table, lens, self.cos, self.sin, qs=q, cu_new=cu_new)
        ctx = coc.kv_cache_attention(q, self.cache, block_table, lens, cu_new=cu_new, window=self.window, sinks=self.sinks)
        return coc.matmul_all_reduce_w4a16([c.view(tokens, hq * d) for c in ctx], self.w_out, self.scales, self.group,
                                           zeros=self.zeros, outs=outs)


class MlpBlock:
    """One layer's gated feed-forward block on R ranks with 8-bit weights: rank r
    holds ffn/R columns of the gate and the up projection and as many rows of
    the down projection.

    norm: hidden values in the activations' type.  w_up[r], up_scales[r]: the
    rank's gate rows, then its up rows (coc.f8_pack with parts=2 of (2 ffn/R) x
    hidden); w_down[r], down_scales[r]: hidden x ffn/R (coc.f8_pack)."""

    def __init__(self, norm, w_up, up_scales, w_down, down_scales, eps: float = 1e-6):
        self.norm, self.eps = norm, eps
        self.w_up, self.up_scales, self.w_down, self.down_scales = w_up, up_scales, w_down, down_scales

    def __call__(self, xs, residuals=None, outs=None, sums=None, stream=None):
        """xs[r], residuals[r]: rank r's rows (any number, the same on every
        rank) x hidden.  Returns (outs, sums): the block's output of the rank's rows,
        and xs + residuals (the residual that goes with it; None without
        residuals).  With a stream everything that is allocated on the way is that stream's."""
        if stream is not None and coc._stream(stream) != torch.cuda.current_stream().cuda_stream:
            now = torch.cuda.current_stream()
            with torch.cuda.stream(coc._as_stream(stream)):
                new = self(xs, residuals, outs=outs, sums=sums)
            for given, ts in ((outs, new[0]), (sums, new[1])):
                if given is None and ts is not None:
                    ts[0].record_stream(now)        # all ranks' are one allocation
            return new
        x, x_scales, sums = coc.add_rms_norm_f8(xs, self.norm, residuals=residuals, eps=self.eps, sums=sums)
        h, h_scales = coc.all_gather_gated_matmul_f8(x, x_scales, self.w_up, self.up_scales)
        return coc.matmul_reduce_scatter_f8(h, h_scales, self.w_down, self.down_scales, outs=outs, dtype=xs[0].dtype), sums


def random_mlp(R: int, hidden: int, ffn: int, dtype=torch.bfloat16, seed: int = 0, device="cuda"):
    """An MlpBlock with random weights."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    f = ffn // R

    def normal(n, k, std):
        return torch.randn(n, k, generator=g, device=device) * std
    up = [coc.f8_pack(normal(2 * f, hidden, hidden ** -0.5), parts=2) for _ in range(R)]
    down = [coc.f8_pack(normal(hidden, f, ffn ** -0.5)) for _ in range(R)]
    norm = (1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(dtype)
    return MlpBlock(norm, *(list(t) for t in zip(*up)), *(list(t) for t in zip(*down)))


def rotation_tables(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """(cos, sin), float32 positions x rot_dim/2, of the angles p * base**(-2j/rot_dim)."""
    freq = base ** (-torch.arange(rot_dim // 2, dtype=torch.float64, device=device) * 2 / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq[None, :]
    return angle.cos().float(), angle.sin().float()


def random_block(R: int, hidden: int, heads: int, kv_heads: int, head_dim: int, pages: int, page_size: int, positions: int,
                 dtype=torch.bfloat16, group: int = 64, seed: int = 0, device="cuda", **kw):
    """An AttentionBlock with random weights and an empty cache."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    hq, hk, d = heads // R, kv_heads // R, head_dim

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)
    w_qkv = [normal(hidden, (hq + 2 * hk) * d, std=hidden ** -0.5) for _ in range(R)]
    codes = [torch.randint(0, 16, (hq * d, hidden), generator=g, device=device) for _ in range(R)]
    scales = [((0.5 + torch.rand(hq * d // group, hidden, generator=g, device=device)) * 0.2 * (heads * d) ** -0.5).to(dtype)
              for _ in range(R)]
    cos, sin = rotation_tables(positions, d, device=device)
    return AttentionBlock(w_qkv, [coc.w4_pack(c) for c in codes], scales, group, hq, hk, d, cos, sin,
                          coc.KVCache.empty(R, pages, page_size, hk, d, device=device), **kw)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--batch", type=int, default=64, help="sequences (a multiple of 8 x ranks)")
    ap.add_argument("--prompt", type=int, default=1024, help="tokens every sequence starts with")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--ffn", type=int, default=0, help="feed-forward size (a multiple of 16 x ranks); 0: no feed-forward block")
    a = ap.parse_args()
    R, B, dev = a.ranks, a.batch, torch.device("cuda")
    per_seq = -(-(a.prompt + a.steps + 1) // a.page)
    block = random_block(R, a.hidden, a.heads, a.kv_heads, a.head_dim, B * per_seq, a.page, a.prompt + a.steps + 1)
    table = torch.randperm(B * per_seq, device=dev).to(torch.int32).view(B, per_seq).contiguous()
    lens = torch.full((B,), a.prompt, dtype=torch.int32, device=dev)
    # prompts: keys and values of all tokens of every sequence in one call
    tokens = B * a.prompt
    xs = [torch.randn(tokens // R, a.hidden, device=dev).to(torch.bfloat16) for _ in range(R)]
    cu = torch.arange(0, tokens + 1, a.prompt, dtype=torch.int32, device=dev)
    qkv = coc.all_gather_matmul(xs, block.w_qkv)
    hq, hk, d = block.q_heads, block.kv_heads, block.head_dim
    coc.kv_cache_append([t[:, hq * d:(hq + hk) * d].view(tokens, hk, d) for t in qkv],
                        [t[:, (hq + hk) * d:].view(tokens, hk, d) for t in qkv], block.cache, table, lens, block.cos, block.sin,
                        cu_new=cu)
    # single-token steps: each replay takes the lengths and inputs that are in the buffers
    x = [torch.randn(B // R, a.hidden, device=dev).to(torch.bfloat16) for _ in range(R)]
    outs = [torch.empty(B, a.hidden, dtype=torch.bfloat16, device=dev) for _ in range(R)]
    lens += 1
    mlp = random_mlp(R, a.hidden, a.ffn) if a.ffn else None
    rows = B // R

    def step():
        y = block(x, table, lens, outs=outs)
        if mlp is not None:
            mlp([t[r * rows:(r + 1) * rows] for r, t in enumerate(y)], residuals=x)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
        lens += 1
    end.record()
    torch.cuda.synchronize()
    coc.sync_status()
    print(f"{a.steps} steps of {B} sequences from {a.prompt} tokens on {R} ranks: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a step")


if __name__ == "__main__":
    main()
