"""The feed-forward block from the 8-bit operators, each stage against 64 bits from what the stage before it left; the
block in captured graphs, on other streams and in threads; and the binding of its operators."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from tensor_matmul_collective_gb300 import coc
from tensor_matmul_collective_gb300 import decode_step as ds

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
SIZES = [(1, 1, 272, 144, BF), (2, 3, 512, 2 * 272, BF), (4, 16, 256, 4 * 128, HF), (8, 40, 640, 8 * 144, BF), (2, 300, 384, 2 * 400, BF)]


def rows(R, n, h, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(n, h, generator=g)).to(dt).to(DEV) for _ in range(R)]


def joined(ts, dt):
    return torch.cat([t.view(torch.uint8) for t in ts]).view(dt)


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("R,n,hidden,ffn,dt", SIZES)
def test_stages(R, n, hidden, ffn, dt, res):
    mlp = ds.random_mlp(R, hidden, ffn, dtype=dt, seed=n)
    xs, rs = rows(R, n, hidden, dt, 1), rows(R, n, hidden, dt, 2) if res else None
    outs, sums = mlp(xs, rs)
    coc.sync_status()
    # the stages by themselves: the same bits
    c, s, u = coc.add_rms_norm_f8(xs, mlp.norm, residuals=rs, eps=mlp.eps)
    h, hs = coc.all_gather_gated_matmul_f8(c, s, mlp.w_up, mlp.up_scales)
    y = coc.matmul_reduce_scatter_f8(h, hs, mlp.w_down, mlp.down_scales, dtype=dt)
    assert all(torch.equal(a, b) for a, b in zip(y, outs)) and (not res or all(torch.equal(a, b) for a, b in zip(u, sums)))
    eps = float(torch.tensor(mlp.eps))
    for r in range(R):
        total = xs[r].double().cpu() + (rs[r].double().cpu() if res else 0.0)
        want = total / torch.sqrt((total * total).mean(1, keepdim=True) + eps) * mlp.norm.double().cpu()
        f8.check_codes(c[r], s[r], want, 2.0 ** -18 * want.abs(), "norm")       # as in test_gpu_f8_rows.py
    xa, sa, f = joined(c, f8.E4M3), joined(s, f8.E8M0), ffn // R
    for r in range(R):
        g, gsize = f8.product([xa], [sa], [mlp.w_up[r][:f]], [mlp.up_scales[r][:f8.blocks(f)]])
        w, wsize = f8.product([xa], [sa], [mlp.w_up[r][f:]], [mlp.up_scales[r][f8.blocks(f):]])
        silu, ge, we = g * torch.sigmoid(g), f8.sum_error(gsize, hidden), f8.sum_error(wsize, hidden)
        f8.check_codes(h[r], hs[r], silu * w, 1.1 * ge * (w.abs() + we) + silu.abs() * we + 2.0 ** -18 * (silu * w).abs() + 2.0 ** -120, "gated")
    ref, size = f8.product(h, hs, mlp.w_down, mlp.down_scales)
    e, unit = f8.sum_error(size, ffn), 2.0 ** -8 if dt == BF else 2.0 ** -11
    assert ((torch.cat(outs).double().cpu() - ref).abs() <= unit * (ref.abs() + e) + e + 2.0 ** -25).all()


def test_whole_layer_step_runs():
    """Attention, then the feed-forward block on its rows, as the module's command does; two steps give finite values that change."""
    R, hidden, B, page = 2, 256, 16, 16
    block = ds.random_block(R, hidden, 8, 4, 64, pages=2 * B, page_size=page, positions=40, seed=1)
    mlp = ds.random_mlp(R, hidden, 512, seed=2)
    table = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    x, seen = rows(R, B // R, hidden, BF, 5), []
    for _ in range(2):
        y = block(x, table, lens)
        x, _ = mlp([t[r * B // R:(r + 1) * B // R] for r, t in enumerate(y)], residuals=x)
        lens += 1
        seen.append(torch.cat(x).float())
    coc.sync_status()
    assert all(t.isfinite().all() for t in seen) and not torch.equal(*seen)


def native(monkeypatch, on):
    if on:
        assert coc._marshal(), "the compiled marshalling was not built"
    else:
        monkeypatch.setattr(coc, "_native", False)
        monkeypatch.setattr(coc, "_marshal", lambda: False)


def everything(R=2, n=5, hidden=272, ffn=544, dt=BF, **kw):
    """All calls of one small layer and their outputs as bytes."""
    mlp = ds.random_mlp(R, hidden, ffn, dtype=dt, seed=3)
    xs, rs = rows(R, n, hidden, dt, 1), rows(R, n, hidden, dt, 2)
    torch.cuda.synchronize()
    c, s, u = coc.add_rms_norm_f8(xs, mlp.norm, residuals=rs, **kw)
    c0, s0, none = coc.add_rms_norm_f8(xs, mlp.norm, **kw)
    assert none is None
    q, qs = coc.quantize_f8(xs, **kw)
    h, hs = coc.all_gather_gated_matmul_f8(c, s, mlp.w_up, mlp.up_scales, **kw)
    ar = coc.matmul_all_reduce_f8(h, hs, mlp.w_down, mlp.down_scales, dtype=dt, **kw)
    rs_ = coc.matmul_reduce_scatter_f8(h, hs, mlp.w_down, mlp.down_scales, dtype=dt, **kw)
    ag = coc.all_gather_matmul_f8(c, s, mlp.w_up, [t.view(torch.uint8).view(f8.E8M0) for t in _whole_scales(mlp)], dtype=dt, **kw)
    torch.cuda.synchronize()
    for a, b in zip(ar[0].chunk(R), rs_):
        assert torch.equal(a, b)
    return [t.cpu().view(torch.uint8) for ts in (c, s, u, c0, s0, q, qs, h, hs, ar, rs_, ag) for t in ts]


def _whole_scales(mlp):
    """The same weight's scales with blocks that run through: the first ones (their values do not matter here)."""
    n = mlp.w_up[0].shape[0]
    return [t[:f8.blocks(n)].contiguous() for t in mlp.up_scales]


@pytest.mark.parametrize("dt", [BF, HF])
def test_both_marshallings_agree(monkeypatch, dt):
    native(monkeypatch, True)
    first = everything(R=2, n=10, dt=dt)
    native(monkeypatch, False)
    second = everything(R=2, n=10, dt=dt)
    assert len(first) == len(second) and all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.parametrize("on", [True, False])
def test_refusals_of_the_binding(monkeypatch, on):
    native(monkeypatch, on)
    mlp = ds.random_mlp(2, 256, 512)
    x = rows(2, 4, 256, BF, 1)
    c, s = coc.quantize_f8(x)
    calls = [coc.matmul_all_reduce_f8, coc.all_gather_matmul_f8]
    w, ws = mlp.w_down, mlp.down_scales             # 256 x 256
    for call in calls:
        for bad in ([c, s, w, ws[:1]], [c[:1], s, w, ws], [c, [t[:, :1].contiguous() for t in s], w, ws], [[t[:, :128] for t in c], s, w, ws],
                    [c, s, w, [ws[0][:1], ws[1]]]):
            with pytest.raises((ValueError, TypeError)):
                call(*bad)
        with pytest.raises(TypeError):
            call(c, [t.view(torch.uint8) for t in s], w, ws)
        with pytest.raises(TypeError):
            call(x, s, w, ws)
        with pytest.raises(TypeError):
            call(c, s, w, ws, dtype=torch.float32)
        with pytest.raises((ValueError, TypeError)):
            call(c, s, w, ws, outs=[torch.empty(1, 256, dtype=BF, device=DEV)] * 2)
    with pytest.raises((ValueError, TypeError)):
        coc.quantize_f8([t.float() for t in x])
    with pytest.raises(ValueError):
        coc.quantize_f8([t.t() for t in x])
    with pytest.raises(ValueError):
        coc.add_rms_norm_f8(x, mlp.norm[:128])
    with pytest.raises(ValueError):
        coc.add_rms_norm_f8(x, mlp.norm, sums=x)
    with pytest.raises((ValueError, TypeError)):
        coc.add_rms_norm_f8(x, mlp.norm, residuals=x[:1])
    for eps in (0.0, float("nan")):
        with pytest.raises(coc.CocError):
            coc.add_rms_norm_f8(x, mlp.norm, eps=eps)
    with pytest.raises(coc.CocError):
        coc.matmul_reduce_scatter_f8([t[:3] for t in c], [t[:3] for t in s], w, ws)          # 3 rows on 2 ranks
    with pytest.raises(coc.CocError):
        coc.quantize_f8([torch.zeros(2, 24, dtype=BF, device=DEV)])                          # rows of 24 codes
    with pytest.raises(ValueError):
        coc.all_gather_gated_matmul_f8(c, s, [t[:255] for t in w], ws)
    coc.sync_status()


@pytest.mark.parametrize("on", [True, False])
def test_type_of_given_outputs_is_taken(monkeypatch, on):
    native(monkeypatch, on)
    mlp = ds.random_mlp(1, 256, 256)
    c, s = coc.quantize_f8(rows(1, 4, 256, BF, 1))
    out = [torch.empty(4, 256, dtype=HF, device=DEV)]
    got = coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales, outs=out)
    assert got[0] is out[0] and torch.equal(out[0], coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales, dtype=HF)[0])
    assert coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales)[0].dtype == BF


def test_shards_apart_on_two_streams_and_in_threads():
    """AllGather of shards that lie apart stacks them in the stream's workspace: two streams and two threads at once."""
    R, n, k, cols = 4, 24, 1024, 520
    g = torch.Generator().manual_seed(4)
    w, ws = zip(*[coc.f8_pack(torch.randn(cols, k, generator=g) * k ** -0.5) for _ in range(R)])
    w, ws = [t.to(DEV) for t in w], [t.to(DEV) for t in ws]
    made = []
    for i in range(4):
        c, s = coc.quantize_f8(rows(R, n, k, BF, i))
        c, s = [t.clone() for t in c], [t.clone() for t in s]
        made.append((c, s, [t.clone() for t in coc.all_gather_matmul_f8(c, s, w, ws)]))
    torch.cuda.synchronize()
    bad = []

    def work(i, stream):
        for _ in range(30):
            c, s, want = made[i]
            with torch.cuda.stream(stream):
                got = coc.all_gather_matmul_f8(c, s, w, ws)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(i)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(i, st)) for i, st in enumerate((one, two, one, two))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    coc.sync_status()
    assert not bad


def test_no_allocation_after_the_first_calls():
    """The library's own memory: stacked shards take the stream's workspace, everything else none."""
    R, n, hidden = 4, 10, 512
    mlp = ds.random_mlp(R, hidden, 1024)
    w, ws = zip(*[coc.f8_pack(torch.randn(264, hidden, device=DEV)) for _ in range(R)])
    xs = rows(R, n, hidden, BF, 1)

    def calls():
        mlp(xs, xs)
        c, s = coc.quantize_f8(xs)
        coc.all_gather_matmul_f8([t.clone() for t in c], [t.clone() for t in s], list(w), list(ws))
    calls()
    torch.cuda.synchronize()
    before = coc.alloc_count()
    for _ in range(5):
        calls()
    coc.sync_status()
    assert coc.alloc_count() == before


def test_block_on_a_given_stream():
    mlp = ds.random_mlp(2, 512, 1024)
    xs, rs = rows(2, 9, 512, BF, 1), rows(2, 9, 512, BF, 2)
    want, wsum = mlp(xs, rs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for _ in range(20):
            got, gsum = mlp(xs, rs, stream=stream)
            torch.cuda.current_stream().wait_stream(side)
            assert all(torch.equal(a, b) for a, b in zip(got + gsum, want + wsum))
            del got, gsum
    codes, scales = coc.quantize_f8(xs, stream=side)
    side.synchronize()
    assert torch.equal(codes[0].view(torch.uint8), coc.quantize_f8(xs)[0][0].view(torch.uint8))


@pytest.mark.parametrize("n", [3, 200])
def test_two_graphs_of_the_block(n):
    """Captured with shards apart (scratch) and together; replayed with new inputs, in turns and on two streams."""
    R, hidden = 2, 384
    mlp = ds.random_mlp(R, hidden, 768)
    wq, wqs = zip(*[coc.f8_pack(torch.randn(264, hidden, device=DEV) * 0.05) for _ in range(R)])
    graphs = []
    for i in range(2):
        xs, rs = rows(R, n, hidden, BF, 10 + i), rows(R, n, hidden, BF, 20 + i)
        c, s = coc.quantize_f8(xs)
        c, s = [t.clone() for t in c], [t.clone() for t in s]

        def run(xs=xs, rs=rs, c=c, s=s):
            coc.quantize_f8(xs, outs=c, scales=s)
            return mlp(xs, rs), coc.all_gather_matmul_f8(c, s, list(wq), list(wqs))
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            (outs, sums), ag = run()
        graphs.append((graph, xs, rs, run, outs, sums, ag, torch.cuda.Stream()))
    for round_ in range(3):
        wants = []
        for i, (graph, xs, rs, run, *_rest) in enumerate(graphs):
            for a, b in zip(xs + rs, rows(R, n, hidden, BF, 100 + 10 * round_ + i) + rows(R, n, hidden, BF, 200 + round_)):
                a.copy_(b)
            (o, u), ag = run()
            wants.append([t.clone() for t in [*o, *u, *ag]])
        torch.cuda.synchronize()
        for graph, *_r, stream in graphs:
            with torch.cuda.stream(stream):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        coc.sync_status()
        for (graph, xs, rs, run, outs, sums, ag, stream), want in zip(graphs, wants):
            assert all(torch.equal(a, b) for a, b in zip([*outs, *sums, *ag], want))


FIRST_USE = """
import torch
from tensor_matmul_collective_gb300 import coc, decode_step as ds
coc.quantize_f8([torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")])      # the device's state
mlp = ds.random_mlp(2, 256, 512)
for n in (1, 40, 300):
    xs = [torch.randn(n, 256, device="cuda").to(torch.bfloat16) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, sums = mlp(xs, residuals=xs)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    want, _ = mlp(xs, residuals=xs)
    coc.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), n
print("same")
"""


def test_kernels_used_first_in_a_capture():
    """Sizes whose kernels no eager call has run yet are captured, in a process of their own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0 and "same" in done.stdout, done.stdout + done.stderr


@pytest.mark.parametrize("tile", ["0", "1"])
def test_scales_at_odd_addresses(monkeypatch, tile):
    """Scales have no alignment: the same values 0 to 3 bytes into a buffer, rows of whole words."""
    monkeypatch.setenv("COC_F8_TILE", tile)
    n, k, cols = 70, 1024, 264
    c, s = coc.quantize_f8(rows(1, n, k, BF, 1))
    w, ws = coc.f8_pack(torch.randn(cols, k, device=DEV) * 0.03)
    want = coc.matmul_all_reduce_f8(c, s, [w], [ws])[0]

    def moved(t, by):
        buf = torch.zeros(t.numel() + 8, dtype=torch.uint8, device=DEV)
        new = buf[by:by + t.numel()].view(f8.E8M0).view(t.shape)
        new.view(torch.uint8).copy_(t.view(torch.uint8))
        assert new.data_ptr() % 4 == by % 4
        return new
    for by in range(4):
        assert torch.equal(coc.matmul_all_reduce_f8(c, [moved(s[0], by)], [w], [ws])[0], want)
        assert torch.equal(coc.matmul_all_reduce_f8(c, s, [w], [moved(ws, by)])[0], want)


def test_a_chain_of_layers_without_waits():
    """Twenty layers whose kernels each begin before the one before them has ended, against the same layers one at a time."""
    R, n, hidden = 2, 17, 512
    layers = [ds.random_mlp(R, hidden, 1024, seed=i) for i in range(5)]
    xs, rs = rows(R, n, hidden, BF, 1), rows(R, n, hidden, BF, 2)

    def chain(wait):
        x, r = xs, rs
        for i in range(20):
            x, r = layers[i % 5](x, r)
            if wait:
                torch.cuda.synchronize()
        return x
    want = [t.clone() for t in chain(True)]
    for _ in range(5):
        got = chain(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_products_of_every_kind_in_a_row():
    """16-bit, w8A16-like and 8-bit products one after another without waits: kernels that come early share SMs and
    tensor memory with the ones before them."""
    R, hidden = 2, 512
    g = torch.Generator().manual_seed(6)
    w16 = [(torch.randn(hidden, hidden, generator=g) * hidden ** -0.5).to(BF).to(DEV) for _ in range(R)]
    mlps = [ds.random_mlp(R, hidden, f, seed=f) for f in (256, 1024)]
    start = {n: rows(R, n, hidden, BF, n) for n in (8, 40, 264)}

    def chain(x, wait):
        for i in range(12):
            x = coc.matmul_all_reduce(x, w16)
            x = [t.clone() for t in x] if wait else x
            n = x[0].shape[0]
            for mlp in mlps:
                x, _ = mlp([t[:n] for t in x])
            x = coc.all_gather_matmul([t[:n // 8 * 8] for t in x], w16)
            x = [t[:n].contiguous() for t in x]
            if wait:
                torch.cuda.synchronize()
        return x
    for n, x in start.items():
        want = [t.clone() for t in chain(x, True)]
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(chain(x, False), want))
    coc.sync_status()


@pytest.mark.parametrize("tile", ["0", "1"])
def test_nothing_is_written_around_the_outputs(monkeypatch, tile):
    """Outputs in the middle of buffers whose other bytes stay as they were: ragged rows, columns and last blocks."""
    monkeypatch.setenv("COC_F8_TILE", tile)
    R, n, k, f = 2, 131, 272, 144
    mlp = ds.random_mlp(R, k, R * f, seed=1)
    c, s = coc.quantize_f8(rows(R, n, k, BF, 1))
    m, fb, pad = R * n, f8.blocks(f), 4096

    def guarded(rows_, cols, dt):
        size = rows_ * cols * dt.itemsize
        buf = torch.full((size + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)
        return buf, buf[pad:pad + size].view(dt).view(rows_, cols), size
    bufs = [[guarded(m, f, f8.E4M3) for _ in range(R)], [guarded(m, fb, f8.E8M0) for _ in range(R)], [guarded(m, k, BF) for _ in range(R)],
            [guarded(n, k, HF) for _ in range(R)]]
    views = [[b[1] for b in bs] for bs in bufs]
    coc.all_gather_gated_matmul_f8(c, s, mlp.w_up, mlp.up_scales, outs=views[0], scales=views[1])
    coc.matmul_all_reduce_f8(views[0], views[1], mlp.w_down, mlp.down_scales, outs=views[2])
    coc.matmul_reduce_scatter_f8(views[0], views[1], mlp.w_down, mlp.down_scales, outs=views[3])
    coc.sync_status()
    for bs in bufs:
        for buf, _, size in bs:
            assert (buf[:pad] == 0xA5).all() and (buf[pad + size:] == 0xA5).all()
    assert all(torch.equal(v, views[2][0]) for v in views[2])


@pytest.mark.parametrize("inner", [256, 4096])
def test_bounded_wait_reports(monkeypatch, inner):
    """A wait that nothing ends runs out, the call's status says so, and the next call is right again (the test hook, no
    fault); the longer contraction is cut into ranges of a cluster."""
    mlp = ds.random_mlp(1, 256, inner)
    c, s = coc.quantize_f8(rows(1, 40, inner, BF, 1))
    want = coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales)[0].clone()
    for tile in "01":
        monkeypatch.setenv("COC_F8_TILE", tile)
        coc.inject_timeout(True)
        try:
            coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales)
            with pytest.raises(coc.CocError) as e:
                coc.sync_status()
            assert e.value.status == coc.ERR_TIMEOUT
        finally:
            coc.inject_timeout(False)
        assert torch.equal(coc.matmul_all_reduce_f8(c, s, mlp.w_down, mlp.down_scales)[0], want)
        coc.sync_status()
