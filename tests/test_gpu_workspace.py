"""The workspaces of streams: a stream whose handle was another's, the
per-thread default stream, two threads on one stream."""
import ctypes
import threading

import pytest
import torch

from tensor_matmul_collective_gb300 import coc

import kv_util as kv
from gpu_util import DEV
from test_gpu_kv_cache import build, to_cache

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PER_THREAD = 2          # the handle of every thread's own default stream


class Attention:
    """One decode call with a known result, its output given."""

    def __init__(self, length, B=1, seed=1):
        table, rk, rv, qs = build(1, 8, 1, 128, 64, [1] * B, [length] * B, BF, seed)
        self.cache, self.table, self.q = to_cache(rk, rv), table.to(DEV), [x.to(DEV) for x in qs]
        self.lens = torch.full((B,), length, dtype=torch.int32, device=DEV)
        self.want = self(None).clone()

    def __call__(self, stream, out=None):
        out = torch.empty_like(self.q[0]) if out is None else out
        coc.kv_cache_attention(self.q, self.cache, self.table, self.lens, outs=[out], stream=stream)
        return out


class Dispatch:
    """A MoE dispatch: its routing table is in scratch."""

    def __init__(self):
        self.idx = [torch.randint(0, 4, (64,), dtype=torch.int32, device=DEV) for _ in range(2)]
        self.h = [torch.randn(64, 128, device=DEV).to(BF) for _ in range(2)]
        self.w = torch.randn(4, 128, 64, device=DEV).to(BF)
        self.buf = coc.moe_dispatch_grouped_matmul(self.h, self.idx, self.w, 2)
        torch.cuda.synchronize()

    def __call__(self, stream):
        y, xd, counts, offsets = self.buf
        coc.moe_dispatch_grouped_matmul(self.h, self.idx, self.w, 2, xd=xd, y=y, counts=counts, offsets=offsets, stream=stream)


def busy():
    """(stream, event at its end) of some hundred milliseconds of work on a stream of its own."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)
        end = torch.cuda.Event()
        end.record()
    return side, end


def new_stream():
    h = ctypes.c_uint64()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(h))) == 0
    return h.value


def destroy(h):
    assert int(torch.cuda.cudart().cudaStreamDestroy(h)) == 0


def reused(h, tries=64):
    """A new stream with the handle of one that was destroyed, None if the driver gives none."""
    kept = []
    got = None
    for _ in range(tries):
        s = new_stream()
        if s == h:
            got = s
            break
        kept.append(s)
    for s in kept:
        destroy(s)
    return got


def test_reused_handle_waits_for_no_other_stream():
    call = Dispatch()
    a = new_stream()
    call(a)
    torch.cuda.synchronize()
    destroy(a)
    b = reused(a)
    if b is None:
        pytest.skip("no handle came twice")
    side, end = busy()
    call(b)
    assert not end.query(), "the call waited for work of another stream"
    torch.cuda.synchronize()
    destroy(b)
    coc.sync_status()


def test_reused_handle_of_attention():
    one, two = Attention(5000, seed=2), Attention(3000, B=3, seed=3)
    a = new_stream()
    for _ in range(3):
        got1 = one(a)
        torch.cuda.ExternalStream(a).synchronize()
        destroy(a)
        b = reused(a)
        if b is None:
            pytest.skip("no handle came twice")
        got2 = two(b)
        torch.cuda.ExternalStream(b).synchronize()
        assert torch.equal(got1, one.want) and torch.equal(got2, two.want)
        a = b
    destroy(a)
    coc.sync_status()


def in_threads(*fs):
    errors = []

    def guard(f):
        try:
            f()
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=guard, args=(f,)) for f in fs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def test_per_thread_streams_take_turns_without_waiting():
    """Calls on the per-thread default stream from two threads, one after the other: no call waits for the device."""
    one = Attention(5000, seed=2)
    outs = [torch.empty_like(one.q[0]) for _ in range(4)]
    torch.cuda.synchronize()
    turn = [threading.Event() for _ in range(5)]
    waited = []
    end = []

    def thread(k):
        torch.cuda.set_device(0)
        for i in range(k, 4, 2):
            if i:
                turn[i].wait()
            one(PER_THREAD, outs[i])
            if i >= 2:
                waited.append(end[0].query())
            else:
                torch.cuda.synchronize()
            if i == 1:
                end.append(busy()[1])
            turn[i + 1].set()
    in_threads(lambda: thread(0), lambda: thread(1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, one.want) for o in outs)
    assert waited == [False, False]
    coc.sync_status()


def test_two_threads_on_one_stream():
    """Calls of unlike sizes from two threads on one stream, as fast as they come: each has its own result."""
    side = torch.cuda.Stream()
    one, two = Attention(20000, seed=2), Attention(900, B=40, seed=3)
    moe = Dispatch()
    one(side), two(side), moe(side)
    n = 200
    outs = [[torch.empty_like(c.q[0]) for _ in range(n)] for c in (one, two)]
    want = [t.clone() for t in moe.buf[2]]
    torch.cuda.synchronize()
    start = threading.Barrier(3)

    def run(f):
        torch.cuda.set_device(0)
        start.wait()
        for i in range(n):
            f(i)
    in_threads(lambda: run(lambda i: one(side, outs[0][i])), lambda: run(lambda i: two(side, outs[1][i])), lambda: run(lambda i: moe(side)))
    torch.cuda.synchronize()
    for c, got in zip((one, two), outs):
        assert all(torch.equal(o, c.want) for o in got)
    assert all(torch.equal(a, b) for a, b in zip(want, moe.buf[2]))
    coc.sync_status()


def test_a_thread_outgrows_the_workspace_that_another_uses():
    """The smaller buffer is freed behind the other thread's calls, and none of them is between it and its launch."""
    big, small = Attention(20000, seed=2), Attention(500, seed=3)
    for _ in range(3):
        coc.shutdown()
        side = torch.cuda.Stream()
        outs = [[torch.empty_like(c.q[0]) for _ in range(60)] for c in (big, small)]
        torch.cuda.synchronize()
        going = threading.Event()

        def run_small():
            torch.cuda.set_device(0)
            for i in range(60):
                small(side, outs[1][i])
                if i == 20:
                    going.set()

        def run_big():
            torch.cuda.set_device(0)
            going.wait()
            for i in range(60):
                big(side, outs[0][i])
        in_threads(run_small, run_big)
        torch.cuda.synchronize()
        for c, got in zip((big, small), outs):
            assert all(torch.equal(o, c.want) for o in got)
    coc.sync_status()
