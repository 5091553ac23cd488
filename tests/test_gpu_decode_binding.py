"""What the Python binding of the decode-step operators holds on to and checks."""
import pytest
import torch

from tensor_matmul_collective_gb300 import coc

from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def small(R=2):
    cache = coc.KVCache.empty(R, 4, 16, 2, 64)
    x = [torch.zeros(3, 2, 64, dtype=BF, device=DEV) for _ in range(R)]
    tb = torch.arange(3, dtype=torch.int32, device=DEV).view(3, 1)
    return cache, x, tb, torch.ones(3, dtype=torch.int32, device=DEV)


def plain(monkeypatch, native):
    if native:
        assert coc._marshal(), "the compiled marshalling was not built"
    else:
        monkeypatch.setattr(coc, "_native", False)
        monkeypatch.setattr(coc, "_marshal", lambda: False)


@pytest.mark.parametrize("native", [True, False])
def test_cache_of_another_device_is_refused(monkeypatch, native):
    """The addresses of a cache on another GPU never reach a launch: the tensors have to be on the cache's device."""
    plain(monkeypatch, native)
    cache, x, tb, ln = small()
    cache.device = torch.device("cuda", 1)      # where it says its codes are
    with pytest.raises(ValueError):
        coc.kv_cache_append(x, x, cache, tb, ln)
    with pytest.raises(ValueError):
        coc.kv_cache_attention(x, cache, tb, ln)
    coc.sync_status()


def test_cache_tensors_are_fixed():
    """The addresses are stored: neither the lists nor their entries can be exchanged under them."""
    cache, x, tb, ln = small()
    for name in ("k", "v", "k_scale", "v_scale"):
        ts = getattr(cache, name)
        other = torch.empty_like(ts[0])
        held = list(ts)
        with pytest.raises(AttributeError):
            setattr(cache, name, [other, other])
        for change in (lambda: ts.__setitem__(0, other), lambda: ts.__setitem__(slice(0, 1), [other]), lambda: ts.append(other),
                       lambda: ts.pop(), lambda: ts.__delitem__(0), lambda: ts.reverse(), lambda: ts.extend([other]), lambda: ts.clear(),
                       lambda: ts.insert(0, other), lambda: ts.__iadd__([other]), lambda: ts.__imul__(2), lambda: ts.remove(other)):
            with pytest.raises(TypeError):
                change()
        assert len(getattr(cache, name)) == 2 and all(a is b for a, b in zip(getattr(cache, name), held))
        assert [*held] + ts == held + held          # otherwise a list
    coc.kv_cache_append(x, x, cache, tb, ln)
    coc.sync_status()


@pytest.mark.parametrize("native", [True, False])
def test_an_argument_without_a_truth_value_is_the_callers_error(monkeypatch, native):
    plain(monkeypatch, native)
    cache, x, tb, ln = small()
    with pytest.raises(RuntimeError, match="ambiguous"):
        coc.kv_cache_append(x, x, cache, tb, ln, interleaved=torch.zeros(2))
    coc.sync_status()


@pytest.mark.parametrize("native", [True, False])
def test_new_outputs_of_the_ranks_share_one_allocation(monkeypatch, native):
    """As the calls' documentation says, whichever way the arguments are looked at."""
    plain(monkeypatch, native)
    cache, x, tb, ln = small()
    turned = coc.kv_cache_append(x, x, cache, tb, ln, qs=x)
    outs = coc.kv_cache_attention(x, cache, tb, ln)
    w = coc.matmul_all_reduce_w4a16([t.view(3, 128) for t in x], [torch.zeros(16, 24, dtype=torch.int32, device=DEV)] * 2,
                                    [torch.ones(2, 24, dtype=BF, device=DEV)] * 2, 64)
    for ts in (turned, outs, w):
        a, b = ts
        assert a.untyped_storage().data_ptr() == b.untyped_storage().data_ptr()
        assert b.data_ptr() - a.data_ptr() == a.numel() * 2 and a.is_contiguous() and b.is_contiguous()
    coc.sync_status()
