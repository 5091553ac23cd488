"""w4A16 MATMUL_ALL_REDUCE against a float64 product of the same codes, scales and zero points."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def make(R, m, n, ks, group, zeros, dt, seed, zlo=0, zhi=16):
    g = torch.Generator().manual_seed(seed)
    xs = [torch.randn(m, ks, generator=g).to(dt) for _ in range(R)]
    codes = [torch.randint(0, 16, (ks, n), generator=g) for _ in range(R)]
    scales = [(0.001 + 0.009 * torch.rand(ks // group, n, generator=g)).to(dt) for _ in range(R)]
    zs = [torch.randint(zlo, zhi, (ks // group, n), generator=g, dtype=torch.int8) for _ in range(R)] if zeros else None
    return xs, codes, scales, zs


def reference(xs, codes, scales, zs, group):
    """(product, sum of |x| |w|) in float64."""
    y, size = 0.0, 0.0
    for r, x in enumerate(xs):
        z = 8.0 if zs is None else zs[r].double().repeat_interleave(group, 0)
        w = (codes[r].double() - z) * scales[r].double().repeat_interleave(group, 0)
        y = y + x.double() @ w
        size = size + x.double().abs() @ w.abs()
    return y, size


def run(xs, codes, scales, zs, group, **kw):
    return coc.matmul_all_reduce_w4a16([x.to(DEV) for x in xs], [coc.w4_pack(c).to(DEV) for c in codes],
                                       [s.to(DEV) for s in scales], group,
                                       zeros=None if zs is None else [z.to(DEV) for z in zs], **kw)


def check(outs, ref, size, group, K, dt):
    """The output's rounding, and fp32 sums inside a group and over the groups, 2**-23 a step."""
    u = 2.0 ** -8 if dt == BF else 2.0 ** -11
    bound = u * ref.abs() + (group + K / group + 64) * 2.0 ** -23 * size + 2.0 ** -25
    err = (outs[0].cpu().double() - ref).abs()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.2f} of the bound"
    assert all(torch.equal(o, outs[0]) for o in outs)


CASES = [
    # R, m, n, k_shard, group, zeros, dtype
    (1, 1, 8, 32, 32, False, BF),
    (1, 1, 64, 64, 64, True, HF),
    (1, 3, 264, 96, 96, True, BF),
    (2, 8, 1000, 128, 32, False, HF),
    (4, 9, 520, 256, 128, True, BF),
    (8, 16, 256, 1024, 128, False, BF),
    (8, 7, 2056, 160, 32, True, HF),
    (2, 17, 136, 512, 256, True, BF),
    (1, 33, 72, 128, 64, False, HF),
    (1, 100, 328, 256, 64, True, BF),
    (1, 2, 4096, 4096, 128, False, HF),
    (2, 12, 88, 7168, 7168, True, BF),
    (1, 1, 16, 16384, 32, False, BF),
    (8, 1, 8, 32, 32, True, HF),
]


@pytest.mark.parametrize("R,m,n,ks,group,zeros,dt", CASES)
def test_w4_product(R, m, n, ks, group, zeros, dt):
    xs, codes, scales, zs = make(R, m, n, ks, group, zeros, dt, seed=m + n)
    outs = run(xs, codes, scales, zs, group)
    coc.sync_status()
    ref, size = reference(xs, codes, scales, zs, group)
    check(outs, ref, size, group, R * ks, dt)
    again = run(xs, codes, scales, zs, group)
    assert torch.equal(again[0], outs[0])


@pytest.mark.parametrize("dt", [BF, HF])
def test_w4_zero_points_of_any_int8(dt):
    xs, codes, scales, zs = make(2, 5, 72, 128, 32, True, dt, 3, zlo=-128, zhi=128)
    zs[0][0, :4] = torch.tensor([-128, 127, 0, -1], dtype=torch.int8)
    outs = run(xs, codes, scales, zs, 32)
    ref, size = reference(xs, codes, scales, zs, 32)
    check(outs, ref, size, 32, 256, dt)


def test_w4_every_code_in_every_place():
    """x is a unit vector: the outputs are single weights, exact in fp32 and rounded once."""
    n, ks, group = 16, 64, 32
    codes = (torch.arange(ks)[:, None] * 5 + torch.arange(n)[None, :] * 3) % 16
    scales = [(torch.arange(1, 2 * n + 1).view(2, n) / 64.0).to(HF)]
    for k in range(ks):
        x = torch.zeros(1, ks, dtype=HF)
        x[0, k] = 1
        out = run([x], [codes], scales, None, group)[0].cpu().double()
        assert torch.equal(out[0], ((codes[k] - 8).double() * scales[0][k // group].double()).to(HF).double()), k


@pytest.mark.parametrize("dt", [BF, HF])
def test_w4_nan_and_infinite_rows_stay_apart(dt):
    """A row of x with NaN or an infinity leaves the other rows' sums alone."""
    xs, codes, scales, zs = make(1, 6, 40, 64, 32, True, dt, 5)
    bad = xs[0].clone()
    bad[1, 3], bad[4, 40] = float("nan"), float("inf")
    out = run([bad], codes, scales, zs, 32)[0].cpu()
    good = run(xs, codes, scales, zs, 32)[0].cpu()
    keep = [0, 2, 3, 5]
    assert torch.equal(out[keep], good[keep])
    assert out[1].isnan().all()
    assert not out[4].isfinite().any()


def test_w4_empty_and_given_outputs():
    outs = coc.matmul_all_reduce_w4a16([torch.zeros(0, 32, dtype=BF, device=DEV)], [torch.zeros(4, 8, dtype=torch.int32, device=DEV)],
                                       [torch.ones(1, 8, dtype=BF, device=DEV)], 32)
    assert outs[0].shape == (0, 8)
    given = [torch.full((2, 8), float("nan"), dtype=BF, device=DEV) for _ in range(2)]
    got = coc.matmul_all_reduce_w4a16([torch.zeros(2, 0, dtype=BF, device=DEV)] * 2, [torch.zeros(0, 8, dtype=torch.int32, device=DEV)] * 2,
                                      [torch.zeros(0, 8, dtype=BF, device=DEV)] * 2, 32, outs=given)
    coc.sync_status()
    assert got[0] is given[0] and not given[0].any() and not given[1].any()


def test_w4_streams_and_graphs():
    xs, codes, scales, zs = make(2, 4, 1024, 512, 128, False, BF, 9)
    want = run(xs, codes, scales, zs, 128)[0].clone()
    args = [[x.to(DEV) for x in xs], [coc.w4_pack(c).to(DEV) for c in codes], [s.to(DEV) for s in scales], 128]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = coc.matmul_all_reduce_w4a16(*args)[0]
    side.synchronize()
    assert torch.equal(got, want)
    outs = [torch.empty_like(want) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        coc.matmul_all_reduce_w4a16(*args, outs=outs)
    args[0][0].mul_(2.0)
    args[0][1].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], (want.float() * 2).to(BF))


@pytest.mark.parametrize("m,n,ks", [(1, 8, 32), (9, 72, 128), (5, 200, 96)])
def test_w4_nothing_is_written_around_the_outputs(m, n, ks):
    xs, codes, scales, zs = make(1, m, n, ks, 32, True, BF, 8)
    buf = torch.full((m * n + 512,), 7.0, dtype=BF, device=DEV)
    run(xs, codes, scales, zs, 32, outs=[buf[256:256 + m * n].view(m, n)])
    coc.sync_status()
    assert (buf[:256] == 7).all() and (buf[256 + m * n:] == 7).all()


@pytest.mark.parametrize("m", [3, 16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 192, 256, 384])
def test_w4_group_sizes(group, zeros, m):
    """Groups of one stage and of several, in both types; ranges that begin inside a group."""
    for dt in (BF, HF):
        ks = 768 if group != 256 else 1024
        xs, codes, scales, zs = make(2, m, 136, ks, group, zeros, dt, seed=group + m)
        outs = run(xs, codes, scales, zs, group)
        coc.sync_status()
        ref, size = reference(xs, codes, scales, zs, group)
        check(outs, ref, size, group, 2 * ks, dt)


@pytest.mark.parametrize("R,m,n,ks", [(1, 1, 64, 8192), (2, 6, 704, 6528), (1, 12, 512, 7168), (4, 2, 1152, 4096), (8, 8, 2432, 512), (1, 8, 10240, 512)])
def test_w4_few_columns_and_many(R, m, n, ks):
    """One to eight ranges of the contraction a slab; as many slabs as do not fit the SMs at once."""
    xs, codes, scales, zs = make(R, m, n, ks, 64, True, BF, seed=n)
    outs = run(xs, codes, scales, zs, 64)
    coc.sync_status()
    ref, size = reference(xs, codes, scales, zs, 64)
    check(outs, ref, size, 64, R * ks, BF)
    again = run(xs, codes, scales, zs, 64)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))
