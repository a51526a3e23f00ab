"""The K/V cache's entry points without a GPU: bad arguments are refused on the
host, before any CUDA call, with the documented status codes."""
import ctypes as C

import pytest
import torch

P = 0x10000  # a 64 KiB-aligned fake device address: never dereferenced


@pytest.fixture(scope="module")
def nv():
    import block_scale_search_b200 as nv
    from block_scale_search_b200 import _build
    _build.build()
    nv.lib()
    return nv


GOOD = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, k_S=P, v_S=P, num_pages=64,
            code_page_stride=4 * 16 * 64, scale_page_stride=4 * 16 * 8, page_size=16, kv_heads=4,
            head_dim=128)


def desc(nv, **kw):
    d = dict(GOOD, **kw)
    return nv.KVCacheDesc(*[d[n] for n, _ in nv.KVCacheDesc._fields_])


BAD_CACHES = [(dict(k_codes=None), -1), (dict(v_scales=None), -1), (dict(k_S=None), -1),
              (dict(num_pages=0), -1), (dict(kv_heads=0), -1), (dict(head_dim=-16), -1),
              (dict(num_pages=1 << 31), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
              (dict(head_dim=72), -2), (dict(head_dim=2048), -2),
              (dict(code_page_stride=4 * 16 * 64 - 16), -2), (dict(scale_page_stride=0), -2),
              (dict(k_codes=P + 8), -3), (dict(v_scales=P + 4), -3),
              (dict(code_page_stride=4 * 16 * 64 + 8), -3), (dict(k_S=P + 2), -3)]


def calls(L, c):
    r = C.byref(c)
    src = (C.c_int32 * 2)(1, 2)
    dst = (C.c_int32 * 2)(3, 4)
    yield L.nvfp4_kv_append(r, P, P, 0, 4, 512, 128, 512, 128, P, None, None)
    yield L.nvfp4_kv_read(r, P, 4, 0, P, P, None)
    yield L.nvfp4_kv_copy_pages(r, 1, 0, 0, src, dst, 2, None)
    yield L.nvfp4_kv_attention(r, P, 0, 8, 4, 1024, 128, P, P, P, 8, 4, 1, 64, 0.1, 1, 0, P, 1024, 128,
                               None, P, 1 << 30, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_cache(nv, kw, status):
    assert list(calls(nv.lib(), desc(nv, **kw))) == [status] * 4


def test_null_cache(nv):
    L = nv.lib()
    assert L.nvfp4_kv_read(None, P, 4, 0, P, P, None) == -1


def refused(fn, names, ok, cases):
    for kw, status in cases:
        a = dict(zip(names, ok))
        a.update(kw)
        assert fn(*[a[n] for n in names]) == status, (kw, status)


def test_append_refusals(nv):
    names = ["c", "K", "V", "type", "n", "kt", "kh", "vt", "vh", "slots", "status", "stream"]
    ok = (C.byref(desc(nv)), P, P, 0, 4, 512, 128, 512, 128, P, None, None)
    refused(nv.lib().nvfp4_kv_append, names, ok, [
        (dict(K=None), -1), (dict(V=None), -1), (dict(slots=None), -1), (dict(type=3), -1),
        (dict(type=-1), -1), (dict(n=-1), -1), (dict(kt=-8), -1), (dict(vh=-8), -1),
        (dict(n=1 << 41), -2), (dict(kt=1 << 41), -2), (dict(K=P + 8), -3), (dict(kt=516), -3),
        (dict(vh=4), -3), (dict(type=2, kt=514), -3), (dict(slots=P + 4), -3), (dict(status=P + 1), -3),
        (dict(n=0), 0), (dict(n=0, K=None, V=None, slots=None), 0)])


def test_read_refusals(nv):
    names = ["c", "slots", "n", "type", "K", "V", "stream"]
    ok = (C.byref(desc(nv)), P, 4, 0, P, P, None)
    refused(nv.lib().nvfp4_kv_read, names, ok, [
        (dict(slots=None), -1), (dict(K=None), -1), (dict(n=-1), -1), (dict(type=5), -1),
        (dict(K=P + 16), -3), (dict(slots=P + 4), -3), (dict(n=0), 0)])


def test_copy_refusals(nv):
    L, c = nv.lib(), desc(nv)

    def call(src, dst, layers=1, cs=0, ss=0, n=None):
        a = (C.c_int32 * max(1, len(src)))(*src)
        b = (C.c_int32 * max(1, len(dst)))(*dst)
        return L.nvfp4_kv_copy_pages(C.byref(c), layers, cs, ss, a, b, len(src) if n is None else n, None)

    assert call([1, 2], [3, 64]) == -1        # past the cache
    assert call([-1, 2], [3, 4]) == -1
    assert call([64, 2], [3, 4]) == -1
    assert call([1, 2], [-3, 4]) == -1
    assert call([1, 2], [3, 3]) == -1         # written twice
    assert call([1, 2], [2, 3]) == -1         # read and written
    assert call([5], [5]) == -1               # onto itself
    assert call([1], [2], layers=-1) == -1
    assert call([1], [2], n=-1) == -1
    assert call([1], [2], layers=70000) == -2
    assert call([1], [2], layers=2, cs=8, ss=16) == -3
    assert call([1], [2], layers=2, cs=-16, ss=16) == -1
    assert call([], []) == 0                  # nothing to do, no device needed
    assert call([1], [2], layers=0) == 0
    assert L.nvfp4_kv_copy_pages(C.byref(c), 1, 0, 0, None, None, 1, None) == -1


def test_attention_refusals(nv):
    names = ["c", "Q", "type", "heads", "total", "qt", "qh", "off", "len", "table", "ts", "batch", "max_q",
             "max_kv", "scale", "causal", "window", "out", "ot", "oh", "lse", "ws", "wsb", "stream"]
    ok = (C.byref(desc(nv)), P, 0, 8, 4, 1024, 128, P, P, P, 8, 4, 1, 64, 0.1, 1, 0, P, 1024, 128, None, P,
          1 << 40, None)
    refused(nv.lib().nvfp4_kv_attention, names, ok, [
        (dict(Q=None), -1), (dict(out=None), -1), (dict(off=None), -1), (dict(len=None), -1),
        (dict(table=None), -1), (dict(type=2), -1), (dict(total=-1), -1), (dict(batch=-1), -1),
        (dict(max_q=-1), -1), (dict(max_kv=-1), -1), (dict(causal=2), -1), (dict(window=-1), -1),
        (dict(causal=0, window=4), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
        (dict(heads=0), -1), (dict(heads=6), -2), (dict(heads=2048), -2), (dict(batch=65536), -2),
        (dict(max_kv=129), -2), (dict(max_q=1 << 31), -2), (dict(total=1 << 31), -2),
        (dict(c=C.byref(desc(nv, head_dim=32))), -2), (dict(Q=P + 8), -3), (dict(qt=1028), -3),
        (dict(oh=4), -3), (dict(lse=P + 2), -3), (dict(off=P + 2), -3), (dict(ws=None), -7),
        (dict(ws=P + 16), -3), (dict(batch=0), 0), (dict(total=0), 0), (dict(max_q=0), 0)])


def test_workspace_size_refuses(nv):
    f = nv.lib().nvfp4_kv_attention_workspace_size
    assert f(-1, 1, 64, 8, 4, 128) == 0
    assert f(4, 1, 64, 6, 4, 128) == 0
    assert f(4, 1, 64, 8, 4, 96) == 0


def test_python_refusals(nv):
    z = torch.zeros
    with pytest.raises(ValueError):   # CPU tensors
        nv.KVCache(z(2, 4, 16, 64, dtype=torch.uint8), z(2, 4, 16, 8, dtype=torch.uint8),
                   z(2, 4, 16, 64, dtype=torch.uint8), z(2, 4, 16, 8, dtype=torch.uint8), z(4), z(4))
    with pytest.raises(ValueError):   # shapes that do not agree
        nv.KVCache(z(2, 4, 16, 64, dtype=torch.uint8), z(2, 4, 16, 4, dtype=torch.uint8),
                   z(2, 4, 16, 64, dtype=torch.uint8), z(2, 4, 16, 8, dtype=torch.uint8), z(4), z(4))
