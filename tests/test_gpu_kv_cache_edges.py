"""The K/V cache at the ends of its numbers and arguments, on a B200: the default
stream's handle, queries that hold Inf, rows whose elements lie far apart,
weights far below a row's largest, NaN in parts of a row that weigh nothing."""
import pytest
import torch

from test_gpu_kv_cache import BF16, DEV, FP16, build_batch, check, decode, make_cache, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import block_scale_search_b200 as nv
    nv.lib()
    assert torch.cuda.is_available()
    yield nv
    assert nv.nvfp4_debug_kv_stalls() == 0


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# --------------------------------------------------------- queries with Inf

def one_sequence(nv, gen, K, V, Q):
    """A cache that holds rows K, V [tokens, heads, dim], and one sequence's arguments."""
    n, heads, dim = K.shape
    S = torch.full((heads,), 2.0 ** -9, device=DEV)
    pages, table = build_batch(gen, [n], 16)
    cache = nv.KVCache.empty(pages, 16, heads, dim, S, S)
    t = torch.arange(n)
    nv.kv_append(cache, K.to(DEV), V.to(DEV), (table[0, t // 16].long() * 16 + t % 16).to(DEV))
    return cache, Q.to(DEV), ints(0, Q.shape[0]), ints(n), table.to(DEV), Q.shape[0], n


@pytest.mark.parametrize("sign", [1, -1, 0])
@pytest.mark.parametrize("lq,lk", [(1, 1), (1, 300), (70, 70), (70, 300)])
@pytest.mark.parametrize("dim", [64, 128])
def test_inf_in_a_query_gives_nan(nv, sign, lq, lk, dim):
    """K has one sign (or 0) in the query's infinite channel: every score is inf, -inf or NaN, the softmax of none a number."""
    gen = torch.Generator().manual_seed(lq + lk)
    K, V = (torch.randn(lk, 2, dim, generator=gen).to(BF16) for _ in range(2))
    K[..., 5] = sign * (1 + K[..., 5].abs())
    Q = torch.randn(lq, 4, dim, generator=gen).to(BF16)
    args = one_sequence(nv, gen, K, V, Q)
    q = args[1].clone()
    bad = torch.zeros(lq, 4, dtype=torch.bool, device=DEV)
    for i, h, x in ((0, 1, float("inf")), (lq - 1, 2, -float("inf")), (lq // 2, 0, float("inf"))):
        args[1][i, h, 5] = x
        bad[i, h] = True
    out, lse = nv.kv_attention(*args, want_lse=True)
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    # (the running maxima of a warp's rows move together, so other rows may differ in their rounding:
    # both results are within the formula's bounds)
    o, l, to, tl = reference(args[0], q, [lq], [lk], args[4], dim ** -0.5, True, 0)
    o[bad.cpu()], l[bad.cpu()] = float("nan"), float("nan")
    check(lse, l, tl, "lse")
    check(out, o, to, "out")


@pytest.mark.parametrize("dim", [64, 128])
def test_inf_scores_in_few_columns_give_nan(nv, dim):
    """A prompt row whose scores are +inf at tokens 6, 7, 14, 15, .. and -inf at all others."""
    gen = torch.Generator().manual_seed(3)
    K, V = (torch.randn(256, 1, dim, generator=gen).to(BF16) for _ in range(2))
    K[..., 5] = torch.where(torch.arange(256) % 8 >= 6, 2.0, -2.0)[:, None]
    Q = torch.randn(80, 2, dim, generator=gen).to(BF16)
    Q[7, 1, 5] = float("inf")
    args = one_sequence(nv, gen, K, V, Q)
    out, lse = nv.kv_attention(*args, causal=False, want_lse=True)
    bad = torch.zeros(80, 2, dtype=torch.bool, device=DEV)
    bad[7, 1] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(lse), bad)
    assert bool(torch.isfinite(out[~bad]).all())


@pytest.mark.parametrize("lq", [1, 70])
def test_inf_query_that_sees_nothing(nv, lq):
    gen = torch.Generator().manual_seed(4)
    K, V = (torch.randn(20, 2, 64, generator=gen).to(BF16) for _ in range(2))
    cache, Q, off, _, table, _, _ = one_sequence(nv, gen, K, V, torch.full((lq, 4, 64), float("inf")).to(BF16))
    out, lse = nv.kv_attention(cache, Q, off, ints(0), table, lq, 20, want_lse=True)
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


# ------------------------------------------------------------- NaN in the cache

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lq,heads", [(40, 8), (300, 2), (2, 8)])
def test_nan_v_of_no_weight_reaches_the_rows_that_see_it(nv, dim, lq, heads):
    """The NaN token's weight is about 2^-300: 0 in 32 bits, and still 0 NaN = NaN."""
    gen = torch.Generator().manual_seed(5)
    n = 6000
    pages, table = build_batch(gen, [n], 16)
    cache = make_cache(nv, gen, pages, 16, 1, dim, scale_lo=0x38, scale_hi=0x39)
    cache.k_S.fill_(1.0)
    cache.k_codes[..., 0] &= 0xF0
    t = n - lq - 20                                   # a token that every row sees
    cache.k_codes[table[0, t // 16], 0, t % 16, 0] = 7
    Q = torch.randn(lq, heads, dim, generator=gen) * 0.01
    Q[..., 0] = 4.0
    Q = Q.to(BF16).to(DEV)
    args = (cache, Q, ints(0, lq), ints(n), table.to(DEV), lq, n, 300 * 0.6931471805599453 / 24.0)
    good, good_lse = nv.kv_attention(*args, want_lse=True)
    assert bool(torch.isfinite(good).all())
    cache.v_scales[table[0, 100 // 16], 0, 100 % 16, 2] = 0x7F
    out, lse = nv.kv_attention(*args, want_lse=True)
    assert bool(torch.isnan(out[..., 32:48]).all())
    assert torch.equal(out[..., :32], good[..., :32]) and torch.equal(out[..., 48:], good[..., 48:])
    assert torch.equal(lse, good_lse)
# ------------------------------------------------------------------ streams

def test_stream_0_is_the_default_stream(nv):
    """What torch.cuda.default_stream().cuda_stream gives: calls follow the work queued there."""
    assert torch.cuda.default_stream().cuda_stream == 0
    gen = torch.Generator().manual_seed(1)
    S = torch.full((2,), 2e-3, device=DEV)
    slots = torch.arange(32, device=DEV)
    K, V = (torch.randn(32, 2, 64, generator=gen).to(BF16).to(DEV) for _ in range(2))
    Q = torch.randn(1, 4, 64, generator=gen).to(BF16).to(DEV)
    off, lens, table = ints(0, 1), ints(32), ints(0, 1)[None]
    want = nv.KVCache.empty(3, 16, 2, 64, S, S)
    nv.kv_append(want, K, V, slots)
    out_want = nv.kv_attention(want, Q, off, lens, table, 1, 32)
    read_want = nv.kv_read(want, slots)
    got = nv.KVCache.empty(3, 16, 2, 64, S, S)
    x, y, q = torch.zeros_like(K), torch.zeros_like(V), torch.zeros_like(Q)
    x.copy_(x), torch.cuda._sleep(10), torch.cuda.Stream()   # loaded and set up before it counts
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)          # about 0.1 s: what does not wait for it sees zeros
    x.copy_(K), y.copy_(V), q.copy_(Q)
    nv.kv_append(got, x, y, slots, stream=0)
    nv.kv_copy_pages(got, [0], [2], stream=0)
    read = nv.kv_read(got, slots, stream=0)
    out = nv.kv_attention(got, q, off, lens, table, 1, 32, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got.k_codes[:2], want.k_codes[:2]) and torch.equal(got.v_scales[:2], want.v_scales[:2])
    assert torch.equal(got.k_codes[2], want.k_codes[0])
    assert all(torch.equal(a, b) for a, b in zip(read, read_want))
    assert torch.equal(out, out_want)


# ------------------------------------------- query elements that lie far apart

@pytest.mark.parametrize("lq", [1, 70])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind,top,low", [(FP16, 2.0 ** 15, 2.0 ** -5), (FP16, 60000.0, 2.0 ** -9),
                                          (BF16, 2.0 ** 20, 2.0 ** -5), (BF16, 3e38, 3e30)])
def test_small_elements_beside_a_large_one(nv, kind, top, low, dim, lq):
    """A row's large element meets zeros of K: its small ones alone make the scores."""
    gen = torch.Generator().manual_seed(lq + dim)
    kv_len = [150, 333]
    pages, table = build_batch(gen, kv_len, 16)
    cache = make_cache(nv, gen, pages, 16, 2, dim)
    cache.k_codes[..., 0] &= 0xF0
    Q = (torch.randn(2 * lq, 4, dim, generator=gen) * low).to(kind)
    Q[..., 0] = top
    Q = Q.to(DEV)
    scale = 0.05 / low if low < 1 else 0.05e-30 / 3
    out, lse = nv.kv_attention(cache, Q, ints(0, lq, 2 * lq), ints(*kv_len), table.to(DEV), lq, max(kv_len), scale,
                               want_lse=True)
    o, l, to, tl = reference(cache, Q, [lq, lq], kv_len, table, scale, True, 0)
    check(lse, l, tl, "lse")
    check(out, o, to, "out")


# -------------------------------------------------- weights far below the largest

@pytest.mark.parametrize("lq", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bits", [10.0, 16.0, 20.0, 24.4, 25.5, 27.0])
def test_weights_far_below_the_largest(nv, lq, dim, bits):
    """Every 32nd token's score is `bits` powers of two above the others' (spread: a third of
    one), and its V is 0, so that the others are the whole output.

    Bound, per element: P is rounded to FP16 (2^-11 of it; where it is subnormal there, half a
    step of 2^-24 in units in which the largest P is 2^7 or more: 2^-32 of the largest weight, 1
    here, so n 2^-32 max|v| / L), scores and exponentials as in reference(), twice."""
    gen = torch.Generator().manual_seed(int(bits * 10) + lq)
    n, heads, kvh = 4096, 4, 1
    pages, table = build_batch(gen, [n], 16)
    cache = make_cache(nv, gen, pages, 16, kvh, dim, scale_lo=0x38, scale_hi=0x39)
    cache.k_S.fill_(1.0)
    sink = torch.arange(0, n, 32)
    p, r = table[0, sink // 16].long().to(DEV), (sink % 16).to(DEV)
    cache.k_codes[..., 0] &= 0xF0                     # element 0: 0
    cache.k_codes[p, 0, r] = 0
    cache.k_codes[p, 0, r, 0] = 7                     # the sinks': 6, and nothing else
    cache.v_codes[p, 0, r] = 0
    Q = torch.randn(lq, heads, dim, generator=gen) * 0.01
    Q[..., 0] = 4.0
    Q = Q.to(BF16).to(DEV)
    scale = bits * 0.6931471805599453 / 24.0
    out, lse = nv.kv_attention(cache, Q, ints(0, lq), ints(n), table.to(DEV), lq, n, scale, causal=False, want_lse=True)
    t = torch.arange(n)
    ids = table[0, t // 16].long()
    k = decode(cache.k_codes.cpu()[ids, 0, t % 16], cache.k_scales.cpu()[ids, 0, t % 16], cache.k_S[0])
    v = decode(cache.v_codes.cpu()[ids, 0, t % 16], cache.v_scales.cpu()[ids, 0, t % 16], cache.v_S[0])
    q = Q.cpu().double()
    x = q @ k.T * scale
    X = (q.abs() @ k.abs().T * scale).amax(-1, keepdim=True)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - m)
    L = w.sum(-1, keepdim=True)
    d = 2 ** -18 * X + 2 ** -17
    o = w @ v / L
    tol = (w @ v.abs() / L * (2 ** -11 + 2 * d) + n * 2 ** -32 * v.abs().max() / L + o.abs() * 2 ** -8)
    check(out, o, tol, "out")
    check(lse, (m + torch.log(L))[..., 0], (d + (m.abs() + torch.log(L)) * 2 ** -21)[..., 0], "lse")


# ---------------------------------------------------------------- large scores

@pytest.mark.parametrize("lq", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bits", [20, 24, 26, 28, 31, 40, 70, 120])
def test_large_scores(nv, lq, dim, bits):
    """Largest scores of 2^bits, seen by two tokens; the next ones are a third less, whose weights
    are 0 in 64 bits.  So out is the mean of two rows of V: both have the same weight, rounded to
    FP16 (2^-11; its exponent, score - m in FP32, is no whole number), against a sum that is not;
    2^-20 for sums and quotients, and out's own rounding.  lse: 2^-21 of it, as elsewhere, and the
    FP32 product of the factors (2^-22)."""
    gen = torch.Generator().manual_seed(bits)
    n, heads = 1500, 8
    pages, table = build_batch(gen, [n], 16)
    cache = make_cache(nv, gen, pages, 16, 1, dim, scale_lo=0x38, scale_hi=0x39)
    cache.k_codes[...] = 0
    cache.k_codes[..., 0] = torch.randint(0, 7, cache.k_codes.shape[:-1], generator=gen, dtype=torch.uint8).to(DEV)
    top = (700, 1203)
    for t in top:
        cache.k_codes[table[0, t // 16], 0, t % 16, 0] = 7
    cache.k_S.fill_(0.7)
    Q = torch.zeros(lq, heads, dim)
    Q[..., 0] = 3.0
    Q[:, 1::2, 0] = -3.0                               # these heads' largest score is 0
    Q = Q.to(FP16).to(DEV)
    scale = 2.0 ** bits / (3.0 * 6.0 * float(cache.k_S[0].double()))
    out, lse = nv.kv_attention(cache, Q, ints(0, lq), ints(n), table.to(DEV), lq, n, scale, causal=False, want_lse=True)
    v = decode(cache.v_codes.cpu()[table[0, torch.arange(n) // 16].long(), 0, torch.arange(n) % 16],
               cache.v_scales.cpu()[table[0, torch.arange(n) // 16].long(), 0, torch.arange(n) % 16], cache.v_S[0])
    o = ((v[top[0]] + v[top[1]]) / 2).expand(lq, heads // 2, dim)
    A = ((v[top[0]].abs() + v[top[1]].abs()) / 2).expand(lq, heads // 2, dim)
    check(out[:, 0::2], o, A * (2 ** -11 + 2 ** -20) + o.abs() * 2 ** -11 + 1e-7, "out")
    l = torch.full((lq, heads // 2), 2.0 ** bits, dtype=torch.float64)
    check(lse[:, 0::2], l, l * (2 ** -21 + 2 ** -22), "lse")
    zero = cache.k_codes.cpu()[table[0, torch.arange(n) // 16].long(), 0, torch.arange(n) % 16, 0] == 0
    o = v[zero].mean(0).expand(lq, heads // 2, dim)
    A = v[zero].abs().mean(0).expand(lq, heads // 2, dim)
    check(out[:, 1::2], o, A * (2 ** -11 + 2 ** -18) + o.abs() * 2 ** -11 + 1e-7, "out of scores 0")
