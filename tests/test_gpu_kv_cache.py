"""The paged NVFP4 K/V cache on a B200: append against the oracle's bytes, read
and attention against plain 64-bit forms, page copies bit for bit, and the four
used together as a server would."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def nv():
    import block_scale_search_b200 as nv
    nv.lib()
    assert torch.cuda.is_available()
    yield nv
    assert nv.nvfp4_debug_kv_stalls() == 0


# ------------------------------------------------------------- plain forms

GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def e4m3_table():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = float("nan") if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def decode(codes, scales, S):
    """float64 numbers [..., dim] of codes [..., dim/2], scales [..., dim/16]; S broadcast over [...]."""
    codes, scales = codes.cpu(), scales.cpu()
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = e4m3_table()[scales.long()].repeat_interleave(16, -1)
    return GRID[n] * v * S.cpu().double()[..., None]


def make_cache(nv, gen, pages, page, heads, dim, layers=None, scale_lo=40, scale_hi=70):
    """A cache of random codes with scale bytes in [scale_lo, scale_hi)."""
    lead = (pages, heads, page) if layers is None else (layers, pages, heads, page)
    t = []
    for _ in range(2):
        t.append(torch.randint(0, 256, (*lead, dim // 2), generator=gen, dtype=torch.uint8).to(DEV))
        t.append(torch.randint(scale_lo, scale_hi, (*lead, dim // 16), generator=gen, dtype=torch.uint8).to(DEV))
    s = (heads,) if layers is None else (layers, heads)
    S = [(torch.rand(*s, generator=gen) + 0.5).to(DEV) for _ in range(2)]
    return nv.KVCache(t[0], t[1], t[2], t[3], S[0], S[1])


def reference(cache, Q, q_len, kv_len, table, scale, causal, window):
    """Attention in 64 bits on the CPU.  Returns out, lse and the bound of out's
    and lse's errors that the documented arithmetic allows: per row
      X   = max over visible j of scale * sum_d |q_d k_jd| (how large sums get),
      A_d = sum_j p_j |v_jd|
      rounding P to FP16: 2^-11 A + (subnormal P) n 2^-25 max|v|
      scores: FP32 sums of up to 128 products, the factor, the exponent's
      argument and base-2 rescaling: 2^-18 X + 2^-17 absolute, which moves p
      relatively by as much and the quotient by twice that"""
    total, heads, dim = Q.shape
    kvh = cache.kv_heads
    G, page = heads // kvh, cache.page_size
    K = decode(cache.k_codes, cache.k_scales, cache.k_S[None, :, None])
    V = decode(cache.v_codes, cache.v_scales, cache.v_S[None, :, None])
    Qd, table = Q.cpu().double(), table.cpu()
    out = torch.zeros(total, heads, dim, dtype=torch.float64)
    lse = torch.full((total, heads), float("-inf"), dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    row = 0
    for b, (lq, lk) in enumerate(zip(q_len, kv_len)):
        t = torch.arange(lk)
        ids = table[b, t // page].long()
        ok = (ids >= 0) & (ids < K.shape[0])
        for h in range(kvh):
            k = K[ids.clamp(0, K.shape[0] - 1), h, t % page]
            v = V[ids.clamp(0, K.shape[0] - 1), h, t % page]
            for i in range(lq):
                p = lk - lq + i
                see = ok.clone()
                if causal:
                    see &= t <= p
                if window:
                    see &= t > p - window
                if not see.any():
                    continue
                ks, vs = k[see], v[see]
                for g in range(G):
                    q = Qd[row + i, h * G + g]
                    x = ks @ q * scale
                    X = ((ks.abs() @ q.abs()) * abs(scale)).max()
                    m = x.max()
                    w = torch.exp(x - m)
                    L = w.sum()
                    o = (w @ vs) / L
                    d = 2 ** -18 * X + 2 ** -17
                    out[row + i, h * G + g] = o
                    lse[row + i, h * G + g] = m + torch.log(L)
                    A = (w @ vs.abs()) / L
                    tol_o[row + i, h * G + g] = (A * (2 ** -11 + 2 * d) + len(x) * 2 ** -25 * vs.abs().max()
                                                 + o.abs() * torch.finfo(Q.dtype).eps / 2 + 1e-7)
                    tol_l[row + i, h * G + g] = d + (m.abs() + torch.log(L)) * 2 ** -21
        row += lq
    return out, lse, tol_o, tol_l


def check(got, want, tol, what):
    got = got.cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    fine = ~nan & ~inf
    err = (got - want).abs()[fine]
    bad = err > tol[fine]
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err - tol[fine]).max())} over its bound"


def build_batch(gen, kv_len, page, extra=3):
    need = [-(-n // page) for n in kv_len]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(kv_len), max(1, max(need, default=1)) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table


def run_attention(nv, gen, q_len, kv_len, heads, kvh, dim, page, kind, causal=True, window=0, spread=1.0,
                  tweak=None, bounds=None, scale=None):
    pages, table = build_batch(gen, kv_len, page)
    cache = make_cache(nv, gen, pages, page, kvh, dim)
    Q = (torch.randn(sum(q_len), heads, dim, generator=gen) * spread).to(kind).to(DEV)
    if tweak:
        tweak(cache, Q, table)
    off = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    scale = dim ** -0.5 if scale is None else scale
    mq, mk = bounds or (max(q_len), max(kv_len))
    out, lse = nv.kv_attention(cache, Q, off, lens, table.to(DEV), mq, mk, scale, causal, window, want_lse=True)
    torch.cuda.synchronize()
    o, l, to, tl = reference(cache, Q, q_len, kv_len, table, scale, causal, window)
    check(lse, l, tl, "lse")
    check(out, o, to, "out")
    return cache, Q, off, lens, table, out, lse


# ------------------------------------------------------------------ append

def oracle_bytes(orc, x, S):
    """Codes and scales of float32 groups x [n, 16] under S by the oracle's sweep without a window."""
    return orc.sweep_group_f32_list(x, None, float(S), 0, 0)[:2]


def rows_of(gen, shape, kind, how):
    x = torch.randn(*shape, generator=gen)
    if how == "tiny":
        x *= 1e-5
    elif how == "large":
        x *= 3e4 if kind != FP16 else 2e3
    elif how == "ties":   # values that are midpoints and grid values under S = 2^-7
        x = (torch.randint(-16, 17, shape, generator=gen) * 0.25) * 2.0 ** torch.randint(-8, 2, shape[:-1] + (1,), generator=gen)
    elif how == "zeros":
        x *= (torch.rand(*shape, generator=gen) < 0.02)
    return x.to(kind)


@pytest.mark.parametrize("kind", [BF16, FP16, FP32])
@pytest.mark.parametrize("how", ["normal", "tiny", "large", "ties", "zeros"])
def test_append_bytes_equal_the_oracle(nv, orc, kind, how):
    gen = torch.Generator().manual_seed(7)
    heads, dim, page, n = 3, 64, 16, 21
    K, V = (rows_of(gen, (n, heads, dim), kind, how) for _ in range(2))
    S = [2.0 ** -7 if how == "ties" else s for s in (0.0017, 0.4, 3e-4)]
    k_S = torch.tensor(S, device=DEV)
    v_S = torch.tensor(S[::-1], device=DEV)
    cache = nv.KVCache.empty(5, page, heads, dim, k_S, v_S)
    slots = torch.randperm(5 * page, generator=gen)[:n].to(DEV)
    st = torch.full((1,), 99, dtype=torch.int32, device=DEV)
    nv.kv_append(cache, K.to(DEV), V.to(DEV), slots, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    p, r = slots.cpu() // page, slots.cpu() % page
    for X, codes, scales, SS in ((K, cache.k_codes, cache.k_scales, S), (V, cache.v_codes, cache.v_scales, S[::-1])):
        gc, gs = codes.cpu()[p, :, r], scales.cpu()[p, :, r]
        for h in range(heads):
            rc, rs = oracle_bytes(orc, X[:, h].float().reshape(-1, 16).numpy(), np.float32(SS[h]))
            assert np.array_equal(gs[:, h].reshape(-1).numpy(), rs)
            assert np.array_equal(gc[:, h].reshape(-1, 8).numpy(), rc)
        # rows that no slot names stay zero
        used = torch.zeros(5, page, dtype=torch.bool)
        used[p, r] = True
        assert not codes.cpu().permute(0, 2, 1, 3)[~used].any()
        assert not scales.cpu().permute(0, 2, 1, 3)[~used].any()


def test_append_nonfinite_groups(nv):
    K = torch.ones(3, 1, 64, dtype=BF16, device=DEV)
    V = K.clone()
    K[0, 0, 17] = float("inf")
    V[2, 0, 63] = float("nan")
    S = torch.full((1,), 1e-3, device=DEV)
    cache = nv.KVCache.empty(2, 16, 1, 64, S, S)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    nv.kv_append(cache, K, V, torch.tensor([3, 4, 20], device=DEV), st)
    assert int(st) == -5
    assert cache.k_scales[0, 0, 3].tolist()[1] == 0x7F and 0x7F not in cache.k_scales[0, 0, 3].tolist()[::2]
    assert not cache.k_codes[0, 0, 3, 8:16].any()
    assert cache.v_scales[1, 0, 4].tolist()[3] == 0x7F and 0x7F not in cache.v_scales[1, 0, 4].tolist()[:3]
    # in a row that is skipped it does not count
    nv.kv_append(cache, K[:1], V[:1], torch.tensor([-1], device=DEV), st)
    assert int(st) == 0


def test_append_skips_and_strides(nv):
    gen = torch.Generator().manual_seed(3)
    heads, dim, page, n = 2, 128, 32, 50
    qkv = torch.randn(n, 8 + 2 * heads, dim, generator=gen).to(BF16).to(DEV)
    K, V = qkv[:, 8:8 + heads], qkv[:, 8 + heads:]
    S = torch.tensor([0.002, 0.001], device=DEV)
    slots = torch.randperm(4 * page, generator=gen)[:n].to(DEV)
    slots[7], slots[8], slots[49] = -1, 4 * page, 2 ** 40
    a, b = (nv.KVCache.empty(4, page, heads, dim, S, S) for _ in range(2))
    nv.kv_append(a, K, V, slots)
    live = [i for i in range(n) if i not in (7, 8, 49)]
    nv.kv_append(b, K.contiguous()[live], V.contiguous()[live], slots[live])
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, name), getattr(b, name))
    # heads in another order of memory, as a [heads, tokens, dim] projection gives them
    Kt = K.transpose(0, 1).contiguous().transpose(0, 1)
    c = nv.KVCache.empty(4, page, heads, dim, S, S)
    nv.kv_append(c, Kt, V, slots)
    assert torch.equal(c.k_codes, a.k_codes)
    with pytest.raises(nv.NVFP4Error):   # rows that start off a 16-byte boundary
        nv.kv_append(a, torch.empty(n, heads, dim + 4, dtype=BF16, device=DEV)[..., 4:], V, slots)
    with pytest.raises(ValueError):
        nv.kv_append(a, K, V[:-1], slots)
    with pytest.raises(ValueError):
        nv.kv_append(a, K, V, slots.int())
    with pytest.raises(ValueError):
        nv.kv_append(a, K.transpose(1, 2).contiguous().transpose(1, 2), V, slots)


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("dim,heads,page", [(16, 1, 16), (64, 8, 16), (128, 8, 64), (240, 3, 32)])
@pytest.mark.parametrize("n", [1, 37, 700])
def test_read(nv, dim, heads, page, n):
    gen = torch.Generator().manual_seed(n + dim)
    cache = make_cache(nv, gen, 7, page, heads, dim, scale_lo=0, scale_hi=128)   # every byte append writes
    slots = torch.randint(0, 7 * page, (n,), generator=gen)
    slots[n // 2] = -1 if n > 1 else 5
    if n > 4:
        slots[4] = 7 * page
    p, r = slots.clamp(0, 7 * page - 1) // page, slots % page
    hole = (slots < 0) | (slots >= 7 * page)
    want = []
    for codes, scales, S in ((cache.k_codes, cache.k_scales, cache.k_S), (cache.v_codes, cache.v_scales, cache.v_S)):
        w = decode(codes.cpu()[p, :, r], scales.cpu()[p, :, r], S[None, :]).float()
        w[hole] = 0
        want.append(w)
    for kind in (FP32, BF16, FP16):
        got = nv.kv_read(cache, slots.to(DEV), kind)
        for g, w in zip(got, want):
            w = w.to(kind)
            assert torch.equal(torch.isnan(g.cpu()), torch.isnan(w))
            assert torch.equal(g.cpu().nan_to_num(7.0), w.nan_to_num(7.0))
    K = torch.full((n + 1, heads, dim), 9.0, device=DEV)
    V = K.clone()
    nv.kv_read(cache, slots.to(DEV), out=(K[:n], V[:n]))
    assert bool((K[n] == 9).all()) and bool((V[n] == 9).all())


# -------------------------------------------------------------------- copy

@pytest.mark.parametrize("layers,n,page,heads,dim", [(None, 1, 16, 1, 16), (3, 5, 16, 3, 64), (2, 64, 32, 2, 128),
                                                     (1, 65, 16, 8, 128), (2, 1500, 16, 1, 64)])
def test_copy_pages(nv, layers, n, page, heads, dim):
    gen = torch.Generator().manual_seed(n)
    pages = 2 * n + 3
    cache = make_cache(nv, gen, pages, page, heads, dim, layers=layers)
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    src, dst = order[:n].clone(), order[n:2 * n]
    if n > 4:
        src[3] = src[0]     # one page may be copied to several
    want = {}
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        t = getattr(cache, name).cpu().clone()
        pagewise = t if layers is not None else t[None]
        pagewise[:, dst.long()] = pagewise[:, src.long()]
        want[name] = t
    nv.kv_copy_pages(cache, src, dst)
    for name, t in want.items():
        assert torch.equal(getattr(cache, name).cpu(), t), name
    with pytest.raises(nv.NVFP4Error):
        nv.kv_copy_pages(cache, [0, 1], [1, 2])
    nv.kv_copy_pages(cache, [], [])


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", [BF16, FP16])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 1), (10, 2), (16, 4), (16, 1), (32, 1), (6, 6)])
def test_decode(nv, dim, kind, heads, kvh):
    gen = torch.Generator().manual_seed(heads * 100 + kvh + dim)
    kv_len = [1, 15, 16, 17, 0, 33, 100, 257]
    run_attention(nv, gen, [1] * len(kv_len), kv_len, heads, kvh, dim, 16, kind)


@pytest.mark.parametrize("dim,page", [(64, 64), (128, 32), (128, 256)])
@pytest.mark.parametrize("lq", [2, 3, 4, 7, 11, 40])
def test_several_new_tokens(nv, dim, page, lq):
    gen = torch.Generator().manual_seed(lq + page)
    kv_len = [lq, lq + 1, 90, 131, max(0, lq - 2), 0]
    run_attention(nv, gen, [lq] * len(kv_len), kv_len, 8, 2, dim, page, BF16)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 1000])
@pytest.mark.parametrize("lq", [1, 5, 33])
def test_window(nv, window, lq):
    gen = torch.Generator().manual_seed(window + lq)
    kv_len = [300, 64, 47, lq, 129]
    run_attention(nv, gen, [lq] * len(kv_len), kv_len, 4, 2, 128, 16, BF16, window=window)


@pytest.mark.parametrize("lq", [1, 6, 50])
def test_not_causal(nv, lq):
    gen = torch.Generator().manual_seed(lq)
    run_attention(nv, gen, [lq, lq, 0, lq], [70, 3, 12, 0], 8, 2, 64, 16, FP16, causal=False)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompts(nv, dim):
    gen = torch.Generator().manual_seed(dim)
    run_attention(nv, gen, [130, 1, 0, 67, 200], [130, 90, 20, 300, 150], 4, 2, dim, 16, BF16)


@pytest.mark.parametrize("heads,kvh", [(8, 1), (4, 4)])
def test_long_prompt(nv, heads, kvh):
    gen = torch.Generator().manual_seed(heads)
    run_attention(nv, gen, [515, 260], [515, 900], heads, kvh, 128, 64, FP16)


def test_one_long_sequence(nv):
    gen = torch.Generator().manual_seed(5)
    run_attention(nv, gen, [1], [5003], 8, 1, 128, 16, BF16, spread=3.0)


def test_many_ragged_sequences(nv):
    gen = torch.Generator().manual_seed(6)
    kv_len = torch.randint(0, 60, (333,), generator=gen).tolist()
    q_len = [1 if i % 7 else 0 for i in range(333)]
    run_attention(nv, gen, q_len, kv_len, 4, 2, 64, 16, BF16)


def test_bounds_above_the_lengths(nv):
    gen = torch.Generator().manual_seed(8)
    run_attention(nv, gen, [1, 3], [20, 40], 8, 2, 128, 16, BF16, bounds=(9, 48))


@pytest.mark.parametrize("lq", [1, 80])
def test_peaked_and_flat_scores(nv, lq):
    gen = torch.Generator().manual_seed(9)
    run_attention(nv, gen, [lq], [400], 8, 2, 128, 16, BF16, spread=30.0)
    run_attention(nv, gen, [lq], [400], 8, 2, 128, 16, FP16, spread=1e-4)


@pytest.mark.parametrize("lq", [1, 80])
def test_extreme_queries(nv, lq):
    def tweak(cache, Q, table):
        Q[0, 0] = 0                 # a row of zeros
        Q[0, 1] *= 1e-38            # subnormal
        Q[0, 2] *= 1e30             # far outside FP16
        cache.k_S.fill_(1e-32)      # (scores of the last stay small)
    run_attention(nv, torch.Generator().manual_seed(10), [lq, lq], [100, 333], 8, 2, 128, 16, BF16, tweak=tweak)


@pytest.mark.parametrize("lq", [1, 3, 70])
def test_nan_in_unused_places(nv, lq):
    """NaN scales behind the lengths, in pages no table names and in places that a
    row's mask hides reach only the rows that see them."""
    kv_len = [75, 100, 16]

    def tweak(cache, Q, table):
        page = cache.page_size
        for b, n in enumerate(kv_len):
            for t in range(n, -(-n // page) * page):
                cache.k_scales[table[b, t // page], :, t % page] = 0x7F
                cache.v_scales[table[b, t // page], :, t % page] = 0x7F
        used = set(table.flatten().tolist())
        for p in set(range(cache.k_codes.shape[0])) - used:
            cache.k_scales[p] = 0x7F
            cache.v_scales[p] = 0x7F
        # the last token's V, seen by the last query only; part of a row of K at the second last
        cache.v_scales[table[0, 74 // page], :, 74 % page, 1] = 0x7F
        if lq > 1:
            cache.k_scales[table[1, 98 // page], 0, 98 % page, 2] = 0x7F

    gen = torch.Generator().manual_seed(11)
    _, _, _, _, _, out, _ = run_attention(nv, gen, [lq] * 3, kv_len, 4, 2, 64, 16, BF16, tweak=tweak)
    assert bool(torch.isnan(out[lq - 1]).any())
    if lq > 1:
        assert not bool(torch.isnan(out[:lq - 1]).any())


@pytest.mark.parametrize("lq", [1, 3, 70])
def test_nan_before_a_window(nv, lq):
    def tweak(cache, Q, table):
        cache.v_scales[table[0, 0], :, 3] = 0x7F     # seen by no query
        t = 200 - lq - 19                            # seen by the first query only
        cache.v_scales[table[0, t // 16], 0, t % 16, 0] = 0x7F
    run_attention(nv, torch.Generator().manual_seed(12), [lq], [200], 4, 2, 64, 16, BF16, window=20, tweak=tweak)


@pytest.mark.parametrize("lq", [1, 70])
def test_nonfinite_queries_stay_in_their_rows(nv, lq):
    def tweak(cache, Q, table):
        Q[0, 1, 5] = float("inf")
        Q[lq - 1, 3, 0] = float("nan")
    gen = torch.Generator().manual_seed(13)
    pages, table = build_batch(gen, [90], 16)
    cache = make_cache(nv, gen, pages, 16, 2, 64)
    Q = torch.randn(lq, 4, 64, generator=gen).to(BF16).to(DEV)
    off = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
    lens = torch.tensor([90], dtype=torch.int32, device=DEV)
    a = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, 90)
    tweak(cache, Q, table)
    b = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, 90)
    bad = torch.zeros(lq, 4, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[lq - 1, 3] = True
    assert bool(torch.isnan(b[bad]).all())
    assert torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("lq", [1, 70])
def test_bad_pages_hide_their_tokens(nv, lq):
    def tweak(cache, Q, table):
        table[0, 1] = -7
        table[0, 3] = cache.k_codes.shape[0]
        table[1, 0] = 2 ** 31 - 1
    run_attention(nv, torch.Generator().manual_seed(14), [lq, lq], [100, 16 + 70], 4, 2, 64, 16, BF16, tweak=tweak)


@pytest.mark.parametrize("lq", [1, 70])
def test_rows_of_no_sequence_and_strides(nv, lq):
    gen = torch.Generator().manual_seed(15)
    kv_len, heads, dim = [100, 40 + lq], 4, 128
    pages, table = build_batch(gen, kv_len, 16)
    cache = make_cache(nv, gen, pages, 16, 2, dim)
    total = 2 * lq + 3
    wide = torch.randn(total, heads + 3, dim, generator=gen).to(BF16).to(DEV)
    Q = wide[:, 1:1 + heads]
    off = torch.tensor([0, lq, 2 * lq], dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    ref = nv.kv_attention(cache, Q.contiguous()[:2 * lq], off, lens, table.to(DEV), lq, max(kv_len))
    out = torch.full((heads, total, dim), 5.0, dtype=BF16, device=DEV).transpose(0, 1)
    lse = torch.full((total, heads), 5.0, device=DEV)
    got = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, max(kv_len), out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out[:2 * lq], ref)
    assert bool((out[2 * lq:] == 5).all()) and bool((lse[2 * lq:] == 5).all()) and not bool((lse[:2 * lq] == 5).any())


@pytest.mark.parametrize("lq", [1, 70])
def test_lengths_that_break_the_bounds_stay_inside(nv, lq):
    """Offsets and lengths out of range are clamped: nothing outside is touched."""
    gen = torch.Generator().manual_seed(16)
    pages, table = build_batch(gen, [64, 64], 16)
    cache = make_cache(nv, gen, pages, 16, 2, 64)
    Q = torch.randn(2 * lq, 4, 64, generator=gen).to(BF16).to(DEV)
    buf = torch.full((2 * lq + 2, 4, 64), 5.0, dtype=BF16, device=DEV)
    for offs, lens in (([0, 10 ** 6, 10 ** 7], [10 ** 6, -5]), ([-9, lq, 2 * lq], [2 ** 31 - 1, 64]),
                       ([2 * lq, lq, 0], [64, 64])):
        nv.kv_attention(cache, Q, torch.tensor(offs, dtype=torch.int32, device=DEV),
                        torch.tensor(lens, dtype=torch.int32, device=DEV), table.to(DEV), lq, 64,
                        out=buf[:2 * lq])
        torch.cuda.synchronize()
        assert bool((buf[2 * lq:] == 5).all())


def test_attention_python_refusals(nv):
    gen = torch.Generator().manual_seed(17)
    cache = make_cache(nv, gen, 4, 16, 2, 64)
    Q = torch.zeros(1, 4, 64, dtype=BF16, device=DEV)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20], dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    nv.kv_attention(cache, Q, off, lens, table, 1, 20)
    for bad in (dict(Q=Q.float()), dict(Q=Q[..., :32]), dict(Q=Q[0]), dict(q_offsets=off[:1]),
                dict(kv_lengths=lens.long()), dict(page_table=table.long()), dict(max_kv=33),
                dict(out=torch.empty(2, 4, 64, dtype=BF16, device=DEV)), dict(Q=Q.cpu()),
                dict(lse=torch.empty(1, 3, device=DEV))):
        a = dict(Q=Q, q_offsets=off, kv_lengths=lens, page_table=table, max_q=1, max_kv=20)
        a.update(bad)
        with pytest.raises(ValueError):
            nv.kv_attention(cache, **a)
    with pytest.raises(nv.NVFP4Error):   # heads that do not divide
        nv.kv_attention(cache, Q[:, :3].contiguous(), off, lens, table, 1, 20)
    with pytest.raises(nv.NVFP4Error):   # a workspace that is too small
        nv.kv_attention(cache, Q, off, lens, table, 1, 20, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(nv.NVFP4Error):   # a window without a direction
        nv.kv_attention(cache, Q, off, lens, table, 1, 20, causal=False, window=4)
    many = make_cache(nv, gen, 4, 16, 2, 64, layers=2)
    with pytest.raises(ValueError):
        nv.kv_attention(many, Q, off, lens, table, 1, 20)


def test_page_offsets_past_32_bits(nv):
    """Pages 640 MB apart in one 6 GB allocation."""
    gen = torch.Generator().manual_seed(18)
    step, heads, page, dim = 640 << 20, 1, 16, 128
    big = torch.zeros(9 * step, dtype=torch.uint8, device=DEV)

    def view(at, row):
        return torch.as_strided(big, (9, heads, page, row), (step, page * row, row, 1), at)

    S = torch.ones(1, device=DEV)
    cache = nv.KVCache(view(0, 64), view(4096, 8), view(8192, 64), view(12288, 8), S, S)
    K, V = (torch.randn(9 * page, 1, dim, generator=gen).to(BF16).to(DEV) for _ in range(2))
    slots = torch.arange(9 * page, device=DEV).flip(0).contiguous()
    nv.kv_append(cache, K, V, slots)
    small = nv.KVCache.empty(9, page, 1, dim, S, S)
    nv.kv_append(small, K, V, slots)
    assert torch.equal(cache.k_codes, small.k_codes) and torch.equal(cache.v_scales, small.v_scales)
    for a, b in zip(nv.kv_read(cache, slots), nv.kv_read(small, slots)):
        assert torch.equal(a, b)
    table = torch.arange(9, dtype=torch.int32, device=DEV).flip(0).contiguous()[None]
    for lq in (1, 70):
        Q = torch.randn(lq, 2, dim, generator=gen).to(BF16).to(DEV)
        off = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
        lens = torch.tensor([140], dtype=torch.int32, device=DEV)
        assert torch.equal(nv.kv_attention(cache, Q, off, lens, table, lq, 140),
                           nv.kv_attention(small, Q, off, lens, table, lq, 140))
    nv.kv_copy_pages(cache, [8], [0])
    assert torch.equal(cache.k_codes[0], small.k_codes[8]) and torch.equal(cache.v_codes[0], small.v_codes[8])


# ------------------------------------------- streams, graphs, and all together

def decode_state(nv, gen, kv_len, heads=8, kvh=2, dim=128, lq=1):
    pages, table = build_batch(gen, kv_len, 16)
    cache = make_cache(nv, gen, pages, 16, kvh, dim)
    n = len(kv_len)
    Q = torch.randn(lq * n, heads, dim, generator=gen).to(BF16).to(DEV)
    off = (torch.arange(n + 1, dtype=torch.int32) * lq).to(DEV)
    return cache, Q, off, torch.tensor(kv_len, dtype=torch.int32, device=DEV), table.to(DEV)


@pytest.mark.parametrize("lq", [1, 40])
def test_same_bits_every_time_and_on_two_streams(nv, lq):
    gen = torch.Generator().manual_seed(19)
    a = decode_state(nv, gen, [3000, 40, 1500], lq=lq)
    b = decode_state(nv, gen, [77, 2900], lq=lq)
    ra = nv.kv_attention(*a, lq, 3000)
    rb = nv.kv_attention(*b, lq, 2900)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append((nv.kv_attention(*a, lq, 3000, stream=s1), nv.kv_attention(*b, lq, 2900, stream=s2.cuda_stream)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, ra) and torch.equal(y, rb)


@pytest.mark.parametrize("lq", [1, 40])
def test_captured_step_serves_growing_lengths(nv, lq):
    """A captured append + attention, replayed while the sequences grow, equals the calls made eagerly."""
    gen = torch.Generator().manual_seed(20)
    kv_len = [50, 7 + lq, 200]
    cache, Q, off, lens, table = decode_state(nv, gen, [n + 70 for n in kv_len], lq=lq)
    lens.copy_(torch.tensor(kv_len))
    n = lq * 3
    K, V = (torch.randn(n, 2, 128, generator=gen).to(BF16).to(DEV) for _ in range(2))
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    out = torch.empty_like(Q)

    def place():
        for i in range(3):
            for j in range(lq):
                t = kv_len[i] - lq + j
                slots[i * lq + j] = int(table[i, t // 16]) * 16 + t % 16

    def step():
        nv.kv_append(cache, K, V, slots)
        nv.kv_attention(cache, Q, off, lens, table, lq, 270, out=out)

    place()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        kv_len = [x + 9 for x in kv_len]
        lens.copy_(torch.tensor(kv_len))
        Q.copy_(torch.randn(n, 8, 128, generator=gen))
        K.copy_(torch.randn(n, 2, 128, generator=gen))
        place()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(got, out)


def test_serving_run(nv):
    """Two prompts are written and answered, one is forked, both branches go on by
    different tokens; every answer equals plain attention over the numbers that
    the cache holds, and the fork's pages are moved without changing them."""
    gen = torch.Generator().manual_seed(21)
    heads, kvh, dim, page, layers, L = 8, 2, 128, 16, 3, 1
    S = torch.full((layers, kvh), 6.0 / (448 * 6), device=DEV)
    pool = nv.KVCache.empty(40, page, kvh, dim, S, S, layers=layers)
    cache = pool.layer(L)
    table = torch.full((3, 8), -1, dtype=torch.int32)
    table[0, :6] = torch.tensor([5, 9, 2, 30, 31, 17])
    table[1, :2] = torch.tensor([11, 4])
    lens = [83, 20]
    Q, K, V = (torch.randn(sum(lens), h, dim, generator=gen).to(BF16).to(DEV) for h in (heads, kvh, kvh))
    slots = torch.cat([table[b, torch.arange(n) // page].long() * page + torch.arange(n) % page
                       for b, n in enumerate(lens)]).to(DEV)

    def answer(Q, q_len, kv_len, rows):
        t = table[rows].contiguous()
        off = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=DEV)
        ll = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
        out, lse = nv.kv_attention(cache, Q, off, ll, t.to(DEV), max(q_len), max(kv_len), want_lse=True)
        o, l, to, tl = reference(cache, Q, q_len, kv_len, t, dim ** -0.5, True, 0)
        check(out, o, to, "out")
        check(lse, l, tl, "lse")
        return out

    nv.kv_append(cache, K, V, slots)
    answer(Q, lens, lens, [0, 1])
    k, v = nv.kv_read(cache, slots)
    assert (k.cpu().double() - K.cpu().double()).abs().max() < 6 / 8   # the coarsest step is 2 / 6 of a group's largest
    # fork sequence 0: full pages are shared, the last one is copied in every layer
    table[2] = table[0]
    table[2, 5] = 25
    nv.kv_copy_pages(pool, [17], [25])
    lens3 = [84, 84]
    new = torch.tensor([17 * page + 83 % page, 25 * page + 83 % page], device=DEV)
    K2, V2, Q2 = (torch.randn(2, h, dim, generator=gen).to(BF16).to(DEV) for h in (kvh, kvh, heads))
    nv.kv_append(cache, K2, V2, new)
    first = answer(Q2, [1, 1], lens3, [0, 2])
    # compaction: the fork's own page moves to the front
    nv.kv_copy_pages(pool, [25], [0])
    table[2, 5] = 0
    assert torch.equal(answer(Q2, [1, 1], lens3, [0, 2]), first)


# ------------------------------------------------------ larger shapes, at random

def reference_gpu(cache, Q, q_len, kv_len, table, causal, window):
    """reference() for larger shapes: 64 bits on the GPU, a sequence and KV head at a time."""
    total, heads, dim = Q.shape
    kvh, page, scale = cache.kv_heads, cache.page_size, dim ** -0.5
    G = heads // kvh
    out = torch.zeros(total, heads, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((total, heads), float("-inf"), dtype=torch.float64, device=DEV)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    grid, e4m3 = GRID.to(DEV), e4m3_table().to(DEV)

    def rows(codes, scales, S):
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        return grid[n] * e4m3[scales.long()].repeat_interleave(16, -1) * S.double()

    row = 0
    for b, (lq, lk) in enumerate(zip(q_len, kv_len)):
        if lq and lk:
            t = torch.arange(lk, device=DEV)
            ids = table[b].to(DEV)[t // page].long()
            p = (lk - lq + torch.arange(lq, device=DEV))[:, None]
            see = (t <= p) if causal else torch.ones(lq, lk, dtype=torch.bool, device=DEV)
            if window:
                see = see & (t > p - window)
            some = see.any(-1)
            for h in range(kvh):
                k = rows(cache.k_codes[ids, h, t % page], cache.k_scales[ids, h, t % page], cache.k_S[h])
                v = rows(cache.v_codes[ids, h, t % page], cache.v_scales[ids, h, t % page], cache.v_S[h])
                for g in range(G):
                    q = Q[row:row + lq, h * G + g].double()
                    x = (q @ k.T * scale).masked_fill(~see, float("-inf"))
                    X = (q.abs() @ k.abs().T * scale).masked_fill(~see, 0).amax(-1)
                    m = x.amax(-1).masked_fill(~some, 0)
                    w = torch.exp(x - m[:, None])
                    L = w.sum(-1).clamp(min=1e-300)
                    o = w @ v / L[:, None]
                    A = w @ v.abs() / L[:, None]
                    d = 2 ** -18 * X + 2 ** -17
                    at = (slice(row, row + lq), h * G + g)
                    out[at] = o
                    lse[at] = torch.where(some, m + torch.log(L), lse[at])
                    tol_o[at] = (A * (2 ** -11 + 2 * d)[:, None] + see.sum(-1)[:, None] * 2 ** -25 * v.abs().max()
                                 + o.abs() * torch.finfo(Q.dtype).eps / 2 + 1e-7)
                    tol_l[at] = d + (m.abs() + torch.log(L).abs()) * 2 ** -21
        row += lq
    return out.cpu(), lse.cpu(), tol_o.cpu(), tol_l.cpu()


def larger(nv, gen, q_len, kv_len, heads, kvh, dim, page, kind, causal=True, window=0, bounds=None):
    pages, table = build_batch(gen, kv_len, page)
    cache = make_cache(nv, gen, pages, page, kvh, dim)
    Q = torch.randn(sum(q_len), heads, dim, generator=gen).to(kind).to(DEV)
    off = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    mq, mk = bounds or (max(q_len), max(kv_len))
    out, lse = nv.kv_attention(cache, Q, off, lens, table.to(DEV), mq, mk, None, causal, window, want_lse=True)
    o, l, to, tl = reference_gpu(cache, Q, q_len, kv_len, table, causal, window)
    check(lse, l, tl, "lse")
    check(out, o, to, "out")


@pytest.mark.parametrize("dim,heads,kvh,page", [(128, 8, 1, 16), (64, 8, 1, 64), (128, 4, 4, 32)])
@pytest.mark.parametrize("q_len,kv_len", [([65], [9000]), ([300, 0, 40], [5000, 700, 3001]), ([129], [129]),
                                          ([33, 33], [6001, 0])])
def test_few_items_are_split(nv, dim, heads, kvh, page, q_len, kv_len):
    gen = torch.Generator().manual_seed(dim + kv_len[0])
    larger(nv, gen, q_len, kv_len, heads, kvh, dim, page, FP16)
    larger(nv, gen, q_len, kv_len, heads, kvh, dim, page, BF16, window=700)
    larger(nv, gen, q_len, kv_len, heads, kvh, dim, page, BF16, causal=False)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_and_single_tokens_together(nv, dim):
    gen = torch.Generator().manual_seed(30 + dim)
    larger(nv, gen, [1, 700, 1, 33, 1, 9, 0, 257], [4000, 900, 1, 2000, 17, 2500, 30, 257], 8, 2, dim, 16, BF16)


@pytest.mark.parametrize("batch,kvh,heads", [(520, 2, 4), (200, 8, 8), (129, 1, 16), (90, 2, 64)])
def test_many_sequences(nv, batch, kvh, heads):
    """The cut items are joined from a list; batches over 128 are scheduled in steps."""
    gen = torch.Generator().manual_seed(batch)
    kv_len = (torch.randint(0, 700, (batch,), generator=gen) * (torch.rand(batch, generator=gen) < 0.9)).tolist()
    larger(nv, gen, [1] * batch, kv_len, heads, kvh, 64 if batch % 2 else 128, 16, BF16)


@pytest.mark.parametrize("seed", range(30))
def test_random_shapes(nv, seed):
    gen = torch.Generator().manual_seed(1000 + seed)

    def pick(*options):
        return options[int(torch.randint(0, len(options), (1,), generator=gen))]

    kvh, group, dim = pick(1, 2, 3, 5), pick(1, 2, 3, 4, 7, 8, 12, 16), pick(64, 128)
    batch = pick(1, 2, 5, 40)
    most = pick(1, 1, 2, 4, 9, 70, 200) if batch < 40 else pick(1, 2, 5)
    q_len = torch.randint(0, most + 1, (batch,), generator=gen).tolist() if most > 1 else [1] * batch
    q_len[0] = most
    far = pick(30, 300, 3000) if batch < 40 else 400
    kv_len = [int(torch.randint(max(0, n - 3), n + far, (1,), generator=gen)) for n in q_len]
    causal = pick(True, True, True, False)
    larger(nv, gen, q_len, kv_len, kvh * group, kvh, dim, pick(16, 32, 128), pick(BF16, FP16), causal=causal,
           window=pick(0, 0, 1, 17, 250) if causal else 0,
           bounds=(most + pick(0, 3), max(kv_len) + pick(0, 1)) if max(kv_len) else (most, 1))


def test_nan_in_split_prompts(nv):
    """A NaN V in one split's tokens reaches the rows that see it, through the join."""
    gen = torch.Generator().manual_seed(40)
    kv_len, lq, heads, kvh, dim = [5000], 40, 8, 1, 128
    pages, table = build_batch(gen, kv_len, 16)
    cache = make_cache(nv, gen, pages, 16, kvh, dim)
    Q = torch.randn(lq, heads, dim, generator=gen).to(BF16).to(DEV)
    off = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    good = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, 5000)
    t = 5000 - 10                                   # position of query 30
    cache.v_scales[table[0, t // 16], 0, t % 16, 3] = 0x7F
    bad, lse = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, 5000, want_lse=True)
    assert torch.equal(bad[:30], good[:30])
    nan = torch.isnan(bad[30:])
    assert bool(nan[..., 48:64].all()) and not bool(nan[..., :48].any()) and not bool(nan[..., 64:].any())
    assert not bool(torch.isnan(lse).any())
    t = 100
    cache.k_scales[table[0, t // 16], 0, t % 16, 0] = 0x7F
    bad, lse = nv.kv_attention(cache, Q, off, lens, table.to(DEV), lq, 5000, want_lse=True)
    assert bool(torch.isnan(bad).all()) and bool(torch.isnan(lse).all())


def test_captured_page_copies(nv):
    gen = torch.Generator().manual_seed(41)
    cache = make_cache(nv, gen, 12, 16, 2, 64, layers=3)
    src, dst = torch.tensor([1, 2], dtype=torch.int32), torch.tensor([7, 8], dtype=torch.int32)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        nv.kv_copy_pages(cache, src, dst)
    src.fill_(3)                                    # the captured call keeps its own pages
    cache.k_codes.copy_(torch.randint(0, 256, cache.k_codes.shape, generator=gen, dtype=torch.uint8))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.k_codes[:, 7], cache.k_codes[:, 1]) and torch.equal(cache.k_codes[:, 8], cache.k_codes[:, 2])


def test_work_beyond_32_bits_is_refused(nv):
    assert nv.nvfp4_kv_attention_workspace_size(60000, 1, 1 << 20, 64, 64, 128) == 0
    assert nv.nvfp4_kv_attention_workspace_size(60000, 1 << 20, 1 << 10, 64, 64, 128) == 0
    assert nv.nvfp4_kv_attention_workspace_size(1000, 1, 1 << 17, 64, 8, 128) > 0
    cache = make_cache(nv, torch.Generator().manual_seed(0), 4, 16, 64, 128)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_kv_attention(cache.desc, z, 0, 64, 8, 8192, 128, z, z, z, 1 << 16, 60000, 1, 1 << 20, 0.1, 1, 0, z,
                              8192, 128, None, torch.empty(1 << 12, dtype=torch.uint8, device=DEV), 1 << 40)
    assert e.value.status == -2


def test_workspace_elsewhere_is_refused(nv):
    gen = torch.Generator().manual_seed(18)
    cache = make_cache(nv, gen, 4, 16, 2, 64)
    Q = torch.zeros(1, 4, 64, dtype=BF16, device=DEV)
    off, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1], [20]))
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    n = nv.nvfp4_kv_attention_workspace_size(1, 1, 20, 4, 2, 64)
    nv.kv_attention(cache, Q, off, lens, table, 1, 20, workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            nv.kv_attention(cache, Q, off, lens, table, 1, 20, workspace=ws)


@pytest.mark.parametrize("dim,heads,n", [(128, 8, 9001), (16, 1, 120003), (240, 5, 3333), (64, 40, 5002)])
def test_many_tokens_equal_few(nv, dim, heads, n):
    """Calls whose threads take several tokens each, against calls of a few hundred."""
    gen = torch.Generator().manual_seed(n)
    pages = n // 16 + 3
    S = torch.rand(heads, generator=gen).to(DEV) * 1e-3 + 1e-4
    one, few = (nv.KVCache.empty(pages, 16, heads, dim, S, S.flip(0)) for _ in range(2))
    K, V = (torch.randn(n, heads, dim, generator=gen).bfloat16().to(DEV) for _ in range(2))
    slots = torch.randperm(pages * 16, generator=gen)[:n]
    slots[::97] = -1
    slots = slots.to(DEV)
    status = torch.ones(1, dtype=torch.int32, device=DEV)
    nv.kv_append(one, K, V, slots, status)
    for a in range(0, n, 301):
        nv.kv_append(few, K[a:a + 301], V[a:a + 301], slots[a:a + 301])
    assert int(status) == 0
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(few, name)), name
    for kind in (BF16, FP32):
        k, v = nv.kv_read(one, slots, kind)
        for a in range(0, n, 301):
            k1, v1 = nv.kv_read(one, slots[a:a + 301], kind)
            assert torch.equal(k[a:a + 301], k1) and torch.equal(v[a:a + 301], v1), a
