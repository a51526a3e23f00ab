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


def test_rows_that_require_a_gradient_are_refused(nv):
    """The calls have none, and a result without a graph would lose it silently."""
    cache = make_cache(nv, torch.Generator().manual_seed(2), 4, 16, 2, 64)
    K = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    G = K.clone().requires_grad_()
    slots = torch.arange(3, device=DEV)
    Q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    off, lens, table = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1], [3], [[0]]))
    before = cache.k_codes.clone()
    for k, v in ((G, K), (K, G)):
        with pytest.raises(ValueError):
            nv.kv_append(cache, k, v, slots)
    with pytest.raises(ValueError):
        nv.kv_attention(cache, Q, off, lens, table, 1, 3)
    assert torch.equal(cache.k_codes, before)
    with torch.no_grad():
        nv.kv_append(cache, G, G, slots)
        a = nv.kv_attention(cache, Q, off, lens, table, 1, 3)
    nv.kv_append(cache, G.detach(), G.detach(), slots)
    b = nv.kv_attention(cache, Q.detach(), off, lens, table, 1, 3)
    assert torch.equal(a, b) and not a.requires_grad
