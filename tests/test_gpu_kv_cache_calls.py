"""The K/V cache's Python helpers on a B200: calls that would give something else
than they seem to are refused."""
import pytest
import torch

from test_gpu_kv_cache import DEV, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import block_scale_search_b200 as nv
    nv.lib()
    assert torch.cuda.is_available()
    return nv


@pytest.mark.parametrize("layers", [None, 2])
def test_a_cache_keeps_its_tensors(nv, layers):
    """Assigning another tensor would leave the calls on the old one."""
    cache = make_cache(nv, torch.Generator().manual_seed(1), 4, 16, 2, 64, layers=layers)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "k_S", "v_S"):
        t = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, t.clone())
        assert getattr(cache, name) is t
        assert getattr(cache.desc, name) == t.data_ptr()
    for name in ("layers", "device", "desc"):
        with pytest.raises(AttributeError):
            setattr(cache, name, None)
    if layers is None:                      # writing into one is how S is changed
        slots = torch.arange(64, device=DEV)
        k, _ = nv.kv_read(cache, slots)
        cache.k_S.mul_(2)
        k2, _ = nv.kv_read(cache, slots)
        assert torch.equal(k2, 2 * k)
