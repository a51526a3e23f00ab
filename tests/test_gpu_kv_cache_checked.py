"""The K/V cache under the bounds-checked build of the library, on a B200: no
address outside a buffer, and a wait that runs out leaves NaN and a count, never
a number."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WAITS = """
import sys
sys.path.insert(0, "tests")
import torch
import block_scale_search_b200 as nv
from test_gpu_kv_cache import BF16, DEV, build_batch, make_cache

assert nv.lib().nvfp4_debug_checks_compiled()


def call(dim, q_len, kv_len):
    gen = torch.Generator().manual_seed(dim)
    pages, table = build_batch(gen, kv_len, 16)
    cache = make_cache(nv, gen, pages, 16, 1, dim)
    Q = torch.randn(sum(q_len), 4, dim, generator=gen).to(BF16).to(DEV)
    off = torch.tensor([0, *torch.tensor(q_len).cumsum(0).tolist()], dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    return nv.kv_attention(cache, Q, off, lens, table.to(DEV), max(q_len), max(kv_len), want_lse=True)


# few items, split over CTAs; then so many that none is; a sequence of a single token beside them
for dim, q_len, kv_len in ((64, [70, 1], [900, 40]), (128, [300, 1], [2000, 9]),
                           (64, [65] * 160 + [1], [300] * 161), (128, [40] * 160 + [1], [300] * 161)):
    good, good_lse = call(dim, q_len, kv_len)
    assert nv.nvfp4_debug_kv_stalls() == 0
    nv.nvfp4_debug_kv_wait_limit(0)
    bad, lse = call(dim, q_len, kv_len)
    assert nv.nvfp4_debug_kv_stalls(reset=True) > 0
    lost = torch.isnan(lse)       # the others' CTAs got through without a failed look
    assert bool(lost.any()) and not bool(lost[-1].any())
    assert bool(torch.isnan(bad[lost]).all())
    assert torch.equal(bad[~lost], good[~lost]) and torch.equal(lse[~lost], good_lse[~lost])
    print(dim, len(q_len), "rows lost:", int(lost.sum()), "of", lost.numel())
    nv.nvfp4_debug_kv_wait_limit(1 << 32)
    again, lse = call(dim, q_len, kv_len)
    assert nv.nvfp4_debug_kv_stalls() == 0
    assert torch.equal(again, good) and torch.equal(lse, good_lse)
    assert bool(torch.isfinite(good).all())
print("waits ok")
"""


def checked_env():
    from block_scale_search_b200 import _build
    return dict(os.environ, NVFP4HS_LIB=_build.build(checked=True))


def test_a_wait_that_runs_out_leaves_nan():
    """With a limit of 0 cycles a wait is given up at the first look that finds it unfinished."""
    out = subprocess.run([sys.executable, "-c", WAITS], cwd=ROOT, env=checked_env(), capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    assert "waits ok" in out.stdout
    print(out.stdout)


def test_the_normal_build_keeps_its_limit():
    import block_scale_search_b200 as nv
    if nv.lib().nvfp4_debug_checks_compiled():
        pytest.skip("checked build")
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_debug_kv_wait_limit(0)


def test_the_cache_touches_nothing_outside_its_buffers():
    """Every global address of append, read, copy and attention against its buffer's extent."""
    here = os.path.dirname(os.path.abspath(__file__))
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
           os.path.join(here, "test_gpu_kv_cache.py"), os.path.join(here, "test_gpu_kv_cache_edges.py")]
    out = subprocess.run(cmd, cwd=ROOT, env=checked_env(), capture_output=True, text=True, timeout=900)
    tail = out.stdout[-3000:] + out.stderr[-2000:]
    assert out.returncode == 0, tail
    assert "bounds checks: 0 failed" in out.stdout, tail
