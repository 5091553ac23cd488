"""Refusals of the decode-step operators, through the C ABI and the binding, and
the packing of 4-bit codes: nothing here reaches a GPU."""
import ctypes

import pytest
import torch

from tensor_matmul_collective_gb300 import coc

A = 0x7f0000000000
MIS = A + 4


@pytest.fixture(scope="module")
def L():
    from tensor_matmul_collective_gb300 import build
    build.build()
    return coc.lib()


def _arr(vals):
    a = (ctypes.c_void_p * len(vals))()
    for i, v in enumerate(vals):
        a[i] = v
    return a


def _desc(R=2, page_size=64, kv_heads=2, head_dim=128, pages=10, k=A, v=A, ks=A, vs=A):
    d = coc._KVCacheDesc(R=R, page_size=page_size, kv_heads=kv_heads, head_dim=head_dim, pages=pages)
    for r in range(min(max(R, 0), 8)):
        d.k[r], d.v[r], d.k_scale[r], d.v_scale[r] = k, v, ks, vs
    return d


S = (ctypes.c_int64 * 2)(512, 128)


def append(L, d=None, tokens=4, seqs=2, k=None, kstr=S, v=None, vstr=S, hq=4, q=None, qstr=S, qo=None, table=A, width=5, lens=A,
           cu=A, cos=A, sin=A, positions=100, rot=128, dt=1):
    d = _desc() if d is None else d
    p = _arr([A] * 8)
    return L.coc_kv_cache_append(ctypes.addressof(d), tokens, seqs, k or p, kstr, v or p, vstr, hq, q or p, qstr, qo or p, table,
                                 width, lens, cu, cos, sin, positions, rot, 0, dt, None)


def attend(L, d=None, tokens=4, seqs=2, hq=4, q=None, qstr=S, out=None, table=A, width=5, lens=A, cu=A, window=0, sinks=0, dt=1):
    d = _desc() if d is None else d
    p = _arr([A] * 8)
    return L.coc_kv_cache_attention(ctypes.addressof(d), tokens, seqs, hq, q or p, qstr, out or p, table, width, lens, cu, 1.0,
                                    window, sinks, dt, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(L, call):
    for kw, want in ((dict(R=0), coc.ERR_INVALID_ARG), (dict(R=9), coc.ERR_INVALID_ARG), (dict(page_size=48), coc.ERR_SHAPE),
                     (dict(page_size=256), coc.ERR_SHAPE), (dict(head_dim=264), coc.ERR_SHAPE), (dict(head_dim=100), coc.ERR_SHAPE),
                     (dict(head_dim=0), coc.ERR_SHAPE), (dict(kv_heads=0), coc.ERR_SHAPE), (dict(pages=-1), coc.ERR_SHAPE),
                     (dict(k=None), coc.ERR_INVALID_ARG), (dict(v=MIS), coc.ERR_ALIGN), (dict(ks=A + 2), coc.ERR_ALIGN),
                     (dict(vs=None), coc.ERR_INVALID_ARG)):
        assert call(L, _desc(**kw)) == want, kw
    assert call(L, dt=2) == coc.ERR_INVALID_ARG
    assert call(L, tokens=-1) == coc.ERR_SHAPE
    assert call(L, seqs=-1) == coc.ERR_SHAPE
    assert call(L, seqs=0) == coc.ERR_SHAPE
    assert call(L, cu=None) == coc.ERR_SHAPE                # 4 tokens, 2 sequences
    assert call(L, width=-1) == coc.ERR_SHAPE
    assert call(L, lens=None) == coc.ERR_INVALID_ARG
    assert call(L, table=None) == coc.ERR_INVALID_ARG
    assert call(L, lens=A + 2) == coc.ERR_ALIGN
    assert call(L, q=_arr([A, None])) == coc.ERR_INVALID_ARG
    assert call(L, q=_arr([A, MIS])) == coc.ERR_ALIGN
    assert call(L, qstr=(ctypes.c_int64 * 2)(510, 128)) == coc.ERR_ALIGN
    assert call(L, qstr=(ctypes.c_int64 * 2)(-512, 128)) == coc.ERR_SHAPE
    assert call(L, tokens=0, seqs=0, cu=None) == coc.OK     # nothing to do
    assert L.coc_kv_cache_append(None, *[0] * 2, *[None] * 4, 0, *[None] * 4, 0, *[None] * 4, 0, 0, 0, 1, None) == coc.ERR_INVALID_ARG


def test_append_refusals(L):
    assert append(L, hq=-1) == coc.ERR_SHAPE
    assert append(L, cos=None) == coc.ERR_INVALID_ARG
    assert append(L, rot=129) == coc.ERR_SHAPE
    assert append(L, rot=130) == coc.ERR_SHAPE
    assert append(L, rot=0) == coc.ERR_SHAPE
    assert append(L, sin=A + 2) == coc.ERR_ALIGN
    assert append(L, k=_arr([A, None])) == coc.ERR_INVALID_ARG
    assert append(L, v=_arr([MIS, A])) == coc.ERR_ALIGN
    assert append(L, qo=_arr([A, None])) == coc.ERR_INVALID_ARG
    assert append(L, kstr=(ctypes.c_int64 * 2)(512, 4)) == coc.ERR_ALIGN


def test_attention_refusals(L):
    assert attend(L, hq=3) == coc.ERR_SHAPE
    assert attend(L, hq=0) == coc.ERR_SHAPE
    assert attend(L, window=-1) == coc.ERR_INVALID_ARG
    assert attend(L, sinks=4) == coc.ERR_INVALID_ARG        # sinks without a window
    assert attend(L, out=_arr([None, A])) == coc.ERR_INVALID_ARG


def test_w4_refusals(L):
    x = _arr([A] * 2)
    f = L.coc_matmul_all_reduce_w4a16
    assert f(3, 4, 64, 128, x, x, x, None, 64, x, 1, None) == coc.ERR_INVALID_ARG     # ranks
    assert f(2, 4, 64, 128, x, x, x, None, 64, x, 9, None) == coc.ERR_INVALID_ARG     # dtype
    assert f(2, 4, 64, 128, x, x, x, None, 16, x, 1, None) == coc.ERR_SHAPE           # group below 32
    assert f(2, 4, 64, 128, x, x, x, None, 48, x, 1, None) == coc.ERR_SHAPE
    assert f(2, 4, 64, 128, x, x, x, None, 96, x, 1, None) == coc.ERR_SHAPE           # k_shard % group
    assert f(2, 4, 60, 128, x, x, x, None, 64, x, 1, None) == coc.ERR_ALIGN           # n % 8
    assert f(2, 1 << 17, 64, 128, x, x, x, None, 64, x, 1, None) == coc.ERR_SHAPE
    assert f(2, -1, 64, 128, x, x, x, None, 64, x, 1, None) == coc.ERR_SHAPE
    assert f(2, 4, 64, 128, x, _arr([A, None]), x, None, 64, x, 1, None) == coc.ERR_INVALID_ARG
    assert f(2, 4, 64, 128, x, x, _arr([A, MIS]), None, 64, x, 1, None) == coc.ERR_ALIGN
    assert f(2, 4, 64, 128, x, x, x, _arr([None, A]), 64, x, 1, None) == coc.ERR_INVALID_ARG
    assert f(2, 0, 64, 128, x, x, x, None, 64, x, 1, None) == coc.OK
    assert f(2, 4, 0, 128, x, x, x, None, 64, x, 1, None) == coc.OK


def test_w4_pack():
    codes = torch.arange(16 * 24).view(16, 24) * 7 % 16
    words = coc.w4_pack(codes)
    assert words.dtype == torch.int32 and words.shape == (2, 24)
    for i in range(8):
        assert torch.equal((words >> (4 * i)) & 15, codes[i::8].to(torch.int32))
    with pytest.raises(ValueError):
        coc.w4_pack(codes[:9])


def test_binding_refuses_cpu_tensors_and_wrong_types():
    with pytest.raises(ValueError):
        coc.KVCache.empty(1, 2, 16, 1, 32, device="cpu")
    with pytest.raises(TypeError):
        coc.kv_cache_append([], [], None, None, None)
    with pytest.raises(TypeError):
        coc.kv_cache_attention([], None, None, None)
    x = [torch.zeros(1, 32, dtype=torch.bfloat16)]
    with pytest.raises(ValueError):
        coc.matmul_all_reduce_w4a16(x, [torch.zeros(4, 8, dtype=torch.int32)], [torch.zeros(1, 8, dtype=torch.bfloat16)], 32)
