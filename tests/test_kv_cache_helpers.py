"""The K/V cache's Python helpers without a GPU."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def nv():
    import block_scale_search_b200 as nv
    return nv


@pytest.mark.parametrize("ids", [torch.tensor([2 ** 32 + 3]), torch.tensor([-2 ** 32]), torch.tensor([2 ** 31]),
                                 np.array([2 ** 40 + 1]), [2 ** 33], [2 ** 70], [1.5], torch.tensor([1.0]), [True],
                                 torch.tensor([True]), np.array([np.inf]), ["1"], None])
def test_page_ids_that_are_not_32_bit_integers_are_refused(nv, ids):
    """They are refused as such, not taken modulo 2^32 or cut to a whole number."""
    ok = torch.tensor([1], dtype=torch.int32)
    for pair in ((ids, ok), (ok, ids)):
        with pytest.raises(ValueError):
            nv.kv_copy_pages(None, *pair)   # before the cache is looked at


def test_page_ids_of_every_integer_kind(nv):
    for ids in ([3, 9], (3, 9), torch.tensor([3, 9]), np.array([3, 9]), torch.tensor([3, 9], dtype=torch.uint8),
                torch.tensor([3, 0, 9], dtype=torch.int32)[::2], range(3, 10, 6)):
        t = nv._page_ids(ids, "src")
        assert t.dtype is torch.int32 and t.is_contiguous() and t.tolist() == [3, 9]
    assert nv._page_ids([], "src").numel() == 0
    t = torch.tensor([4], dtype=torch.int32)
    assert nv._page_ids(t, "src") is t
