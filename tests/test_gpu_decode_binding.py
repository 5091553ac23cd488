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
