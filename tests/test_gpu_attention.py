"""Exact attention (cross_attention, prefix_attention) against the formula in 64 bits.

Tolerance, element by element.  Products of bf16 values are exact in f32 (those of f32 values
round by 2^-24 each, counted among the sums).  A score is a sum of d products: its rounding
errors are at most 2^-23 of the running sum each (the tensor cores may truncate), so at most
d 2^-23 sum|q_i k_i|; scaling, the subtraction of the reference and the f32 exponent argument
add 3 roundings of 2^-24 (|x| + |m|), x the scaled scores and m their maximum.  An error e of an
exponent moves p by a factor 1 + e, the exponential itself is off by 2^-22, and the normaliser
moves by at most as much: p is off by 2 (e + 2^-22) at most.  Sums over N keys: 6 standard
deviations of N independent roundings, 6 sqrt(N) 2^-23.  All of this scales sum_i p_i |v_i|.
bf16 inputs: each weight is rounded to bf16 for its product, half a step, 2^-8 of it.  At last
y is rounded to its type, half a step of |y| + what it is already off.
lse: the score error, the exponential's, and two roundings of its value.
"""
import math

import pytest
import torch

import sparse_kv_caching_b200 as lola

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    lola.attention_check()


def normal(seed, *shape, dtype=F32, factor=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * factor).to(dtype)


def formula(q, kp, vp, k, v, lens=None, causal=True, scale=None):
    """(y, lse, tolerance of y, tolerance of lse) in 64 bits; kp = None: cross attention."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    y = torch.zeros(B, T, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    ty, tl = torch.zeros_like(y), torch.zeros_like(lse)
    half = torch.finfo(q.dtype).eps / 2
    P = 0 if kp is None else kp.shape[0]
    for b in range(B):
        n = k.shape[1] if lens is None else min(max(int(lens[b]), 0), k.shape[1])
        for t in range(T):
            m = max(0, n - T + t + 1) if causal and kp is not None else n
            if P + m == 0:
                continue
            kk, vv = k[b, :m].double(), v[b, :m].double()
            if P:
                kk, vv = torch.cat([kp.double(), kk]), torch.cat([vp.double(), vv])
            qq = q[b, t].double().view(Hkv, G, d)
            x = torch.einsum("hgd,shd->hgs", qq, kk) * scale
            a = torch.einsum("hgd,shd->hgs", qq.abs(), kk.abs()) * scale
            top = x.max(-1, keepdim=True).values
            p = torch.exp(x - top)
            tot = p.sum(-1, keepdim=True)
            p = p / tot
            N = P + m
            e = (d * 2.0**-23 * a + 3 * 2.0**-24 * (x.abs() + top.abs())).max(-1, keepdim=True).values
            rel = 2 * (e + 2.0**-22) + 6 * math.sqrt(N) * 2.0**-23
            if q.dtype == BF16:
                rel = rel + 2.0**-8
            yy = torch.einsum("hgs,shd->hgd", p, vv)
            off = rel * torch.einsum("hgs,shd->hgd", p, vv.abs())
            y[b, t] = yy.reshape(Hq, d)
            ty[b, t] = (off + half * (yy.abs() + off) + 2.0**-126).reshape(Hq, d)
            ll = top + torch.log(tot)
            lse[b, t] = ll.reshape(Hq)
            tl[b, t] = (e + 2.0**-21 + 6 * math.sqrt(N) * 2.0**-23 + 2 * 2.0**-24 * ll.abs()).reshape(Hq)
    return y, lse, ty, tl


def check(y, lse, want):
    wy, wl, ty, tl = want
    off = (y.double() - wy).abs()
    assert bool((off <= ty).all()), f"y: worst {float((off / ty.clamp_min(1e-300)).max()):.2f} of the tolerance"
    none = torch.isinf(wl)
    assert torch.equal(none, torch.isneginf(lse))
    o, t = (lse.double() - wl).abs()[~none], tl[~none]
    assert bool((o <= t).all()), f"lse: worst {float((o / t).max()):.2f} of the tolerance"


def run_cross(q, k, v, lens=None, **kw):
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    y = lola.cross_attention(q, k, v, kv_len=lens, lse=lse, **kw)
    return y, lse


def run_prefix(q, kp, vp, k, v, lens=None, **kw):
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    y = lola.prefix_attention(q, kp, vp, k, v, own_len=lens, lse=lse, **kw)
    return y, lse


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


CROSS = [  # B, T, S, Hq, Hkv, lengths
    (1, 1, 1, 1, 1, None), (2, 1, 77, 32, 8, None), (3, 1, 128, 8, 8, (0, 1, 128)),
    (4, 1, 700, 28, 4, (700, 129, 127, 64)), (2, 1, 2500, 6, 2, None), (2, 5, 333, 10, 2, (65, 333)),
    (1, 40, 257, 4, 1, None), (3, 33, 130, 3, 1, (130, 0, 17)), (2, 129, 64, 16, 2, (63, 1)),
    (1, 300, 513, 8, 2, None), (2, 64, 1000, 6, 6, (999, 385)), (1, 1, 5, 96, 1, None),
    (2, 7, 300, 64, 1, (300, 200)), (1, 513, 40, 1, 1, None),
]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("B,T,S,Hq,Hkv,lens", CROSS)
def test_cross(dtype, d, B, T, S, Hq, Hkv, lens):
    q, k, v = normal(1, B, T, Hq, d, dtype=dtype), normal(2, B, S, Hkv, d, dtype=dtype), normal(3, B, S, Hkv, d, dtype=dtype)
    n = None if lens is None else ints(*lens)
    check(*run_cross(q, k, v, n), formula(q, None, None, k, v, n))


PREFIX = [  # B, T, P, L, Hq, Hkv, own lengths
    (1, 1, 1, 1, 1, 1, None), (2, 1, 200, 17, 32, 8, None), (5, 1, 513, 40, 8, 2, (40, 0, 1, 39, 7)),
    (3, 1, 0, 100, 4, 4, (100, 33, 1)), (2, 1, 64, 0, 6, 2, None), (33, 1, 130, 3, 12, 4, None),
    (4, 5, 300, 64, 10, 2, (64, 5, 3, 0)), (2, 3, 1, 9, 8, 1, (9, 3)), (2, 70, 129, 200, 4, 2, (200, 70)),
    (3, 40, 257, 40, 6, 2, None), (1, 260, 64, 300, 2, 1, (299,)), (17, 2, 2000, 65, 7, 1, None),
    (2, 130, 0, 130, 4, 2, None), (70, 1, 900, 130, 16, 2, None),
]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("B,T,P,L,Hq,Hkv,lens", PREFIX)
def test_prefix(dtype, d, B, T, P, L, Hq, Hkv, lens):
    q = normal(1, B, T, Hq, d, dtype=dtype)
    kp, vp = normal(2, P, Hkv, d, dtype=dtype), normal(3, P, Hkv, d, dtype=dtype)
    k, v = normal(4, B, L, Hkv, d, dtype=dtype), normal(5, B, L, Hkv, d, dtype=dtype)
    n = None if lens is None else ints(*lens)
    check(*run_prefix(q, kp, vp, k, v, n), formula(q, kp, vp, k, v, n))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 4, 150])
def test_lengths_outside_the_keys_are_clamped(dtype, T):
    q, k, v = normal(1, 3, T, 4, 64, dtype=dtype), normal(2, 3, 90, 2, 64, dtype=dtype), normal(3, 3, 90, 2, 64, dtype=dtype)
    n = ints(-5, 2**31 - 1, 91)
    check(*run_cross(q, k, v, n), formula(q, None, None, k, v, n))
    check(*run_prefix(q, k[0, :50], v[0, :50], k, v, n), formula(q, k[0, :50], v[0, :50], k, v, n))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,G", [(1, 4), (6, 3), (200, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_read_does_not_matter(dtype, T, G, bad):
    """NaN and infinities in keys and values behind each length, and behind the query's own position."""
    B, L, Hkv, d = 3, 333, 2, 128
    q = normal(1, B, T, G * Hkv, d, dtype=dtype)
    k, v = normal(2, B, L, Hkv, d, dtype=dtype), normal(3, B, L, Hkv, d, dtype=dtype)
    kp, vp = normal(4, 70, Hkv, d, dtype=dtype), normal(5, 70, Hkv, d, dtype=dtype)
    n = ints(333, 130, 0)
    want = formula(q, None, None, k, v, n), formula(q, kp, vp, k, v, n)
    for b in range(B):
        k[b, int(n[b]):] = bad
        v[b, int(n[b]):] = bad
    check(*run_cross(q, k, v, n), want[0])
    check(*run_prefix(q, kp, vp, k, v, n), want[1])


@pytest.mark.parametrize("T", [1, 130])
def test_nan_in_a_key_that_is_read_reaches_its_rows_only(T):
    q, k, v = (normal(i, 2, n, 4, 64, dtype=BF16) for i, n in ((1, T), (2, 200), (3, 200)))
    k[1, 77, 2] = math.nan
    y, lse = run_cross(q, k, v)
    assert torch.isnan(y[1, :, 2]).all() and torch.isnan(lse[1, :, 2]).all()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[1, :, [0, 1, 3]]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 3, 140])
def test_large_scores(dtype, T):
    """Scores to +-10^4 and rising along the keys: the running maximum moves at every tile."""
    B, S, H, d = 2, 600, 2, 64
    q = normal(1, B, T, H, d, dtype=dtype, factor=30.0)
    k = (normal(2, B, S, H, d) * torch.linspace(0.1, 30, S, device="cuda")[:, None, None]).to(dtype)
    v = normal(3, B, S, H, d, dtype=dtype)
    check(*run_cross(q, k, v), formula(q, None, None, k, v))
    check(*run_prefix(q, k[0], v[0], k, v), formula(q, k[0], v[0], k, v))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 9, 140])
def test_scale(dtype, T):
    q, k, v = (normal(i, 2, n, 4, 64, dtype=dtype) for i, n in ((1, T), (2, 150), (3, 150)))
    check(*run_cross(q, k, v, scale=0.7), formula(q, None, None, k, v, scale=0.7))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 6, 135])
def test_strides(dtype, T):
    """Keys and values as halves of one projection, queries head-major, a padded cache, one
    encoder output for the batch, one key head for all."""
    B, S, Hq, Hkv, d = 3, 190, 8, 2, 64
    q = normal(1, B, Hq, T, d, dtype=dtype).transpose(1, 2)
    kv = normal(2, B, S, 2, Hkv, d, dtype=dtype)
    k, v = kv[:, :, 0], kv[:, :, 1]
    n = ints(190, 3, 100)
    check(*run_cross(q, k, v, n), formula(q, None, None, k, v, n))
    big = normal(3, B, 400, Hkv, 2 * d, dtype=dtype)
    ko, vo = big[:, 16:16 + S, :, :d], big[:, 16:16 + S, :, d:]
    check(*run_prefix(q, k[0], v[1], ko, vo, n), formula(q, k[0], v[1], ko, vo, n))
    heads = normal(4, B, Hkv, S, d, dtype=dtype).transpose(1, 2)      # head-major cache
    check(*run_cross(q, heads, v, n), formula(q, None, None, heads, v, n))
    one, two = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    check(*run_cross(q, one, two), formula(q, None, None, one, two))
    check(*run_cross(q, one, two, n), formula(q, None, None, one, two, n))
    mq, mv = k[:, :, :1].expand(-1, -1, Hkv, -1), v[:, :, :1].expand(-1, -1, Hkv, -1)
    check(*run_cross(q, mq, mv, n), formula(q, None, None, mq, mv, n))
    q1 = normal(5, 1, T, Hq, d, dtype=dtype).expand(B, -1, -1, -1)     # one query for all sequences
    check(*run_cross(q1, k, v, n), formula(q1, None, None, k, v, n))


def test_offsets_beyond_32_bits():
    """A cache whose last rows lie 2^32 bytes and 2^31 elements behind its first."""
    H, d, S = 2, 64, 2100
    buf = torch.zeros(S, 2**20 // H, H, dtype=BF16, device="cuda").view(S, 2**20)
    rows = normal(1, S, 2, H, d, dtype=BF16)
    k = buf[:, :H * d].view(S, H, d)
    v = buf[:, H * d:2 * H * d].view(S, H, d)
    k.copy_(rows[:, 0])
    v.copy_(rows[:, 1])
    for T in (1, 65):
        q = normal(2, 1, T, 4, d, dtype=BF16)
        check(*run_cross(q, k[None], v[None]), formula(q, None, None, rows[None, :, 0], rows[None, :, 1]))
        check(*run_prefix(q, k, v, k[None], v[None]), formula(q, k, v, k[None], v[None]))


def test_one_key_gives_its_value():
    for dtype in (BF16, F32):
        q, k, v = (normal(i, 2, n, 2, 128, dtype=dtype) for i, n in ((1, 3), (2, 1), (3, 1)))
        assert torch.equal(lola.cross_attention(q, k, v), v.expand(2, 3, 2, 128))


def test_no_keys_at_all():
    for dtype in (BF16, F32):
        for T in (1, 200):
            q, k = normal(1, 2, T, 4, 64, dtype=dtype), torch.empty(2, 0, 2, 64, dtype=dtype, device="cuda")
            y, lse = run_cross(q, k, k)
            assert not y.any() and torch.isneginf(lse).all()
            y, lse = run_prefix(q, k[0], k[0], k, k)
            assert not y.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T", [1, 5, 200])
def test_a_batch_equals_its_sequences(T):
    """Nothing of one sequence depends on another: not even its bits, except that a batch may cut
    the keys at other places (so the tolerance is the formula's)."""
    B, P, L, Hq, Hkv, d = 6, 150, 90, 8, 2, 128
    q, k, v = (normal(i, B, n, h, d, dtype=BF16) for i, n, h in ((1, T, Hq), (2, L, Hkv), (3, L, Hkv)))
    kp, vp = normal(4, P, Hkv, d, dtype=BF16), normal(5, P, Hkv, d, dtype=BF16)
    n = ints(90, 1, 44, 0, 64, 65)
    want = formula(q, kp, vp, k, v, n)
    check(*run_prefix(q, kp, vp, k, v, n), want)
    for b in range(B):
        s = slice(b, b + 1)
        check(*run_prefix(q[s], kp, vp, k[s], v[s], n[s]), tuple(x[s] for x in want))


@pytest.mark.parametrize("T,S", [(1, 5000), (3, 700), (300, 900)])
def test_same_bits_every_time(T, S):
    q, k, v = (normal(i, 4, n, h, 128, dtype=BF16) for i, n, h in ((1, T, 8), (2, S, 2), (3, S, 2)))
    one = [lola.cross_attention(q, k, v), lola.prefix_attention(q, k[0], v[0], k, v)]
    for _ in range(5):
        two = [lola.cross_attention(q, k, v), lola.prefix_attention(q, k[0], v[0], k, v)]
        assert all(torch.equal(x, y) for x, y in zip(one, two))


@pytest.mark.parametrize("T", [1, 150])
def test_side_stream_and_own_buffers(T):
    q, k, v = (normal(i, 2, n, h, 128, dtype=BF16) for i, n, h in ((1, T, 8), (2, 800, 2), (3, 800, 2)))
    want = formula(q, None, None, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = torch.empty(lola.attention_workspace(q, k), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert lola.cross_attention(q, k, v, y=y, lse=lse, workspace=ws, stream=side) is y
    side.synchronize()
    check(y, lse, want)


@pytest.mark.parametrize("T", [1, 4, 150])
def test_captured_and_replayed_with_other_lengths(T):
    B, P, L, Hq, Hkv, d = 3, 700, 400, 8, 2, 128
    q, k, v = (normal(i, B, n, h, d, dtype=BF16) for i, n, h in ((1, T, Hq), (2, L, Hkv), (3, L, Hkv)))
    kp, vp = normal(4, P, Hkv, d, dtype=BF16), normal(5, P, Hkv, d, dtype=BF16)
    n = ints(L, L, L)
    graphs = []
    for _ in range(2):                          # two graphs, each with scratch of its own
        lola.prefix_attention(q, kp, vp, k, v, own_len=n)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = lola.prefix_attention(q, kp, vp, k, v, own_len=n)
            z = lola.cross_attention(q, k, v, kv_len=n)
        graphs.append((g, y, z))
    for lens in ((L, 1, 0), (200, 399, 128)):
        n.copy_(ints(*lens))
        q.copy_(normal(sum(lens), *q.shape, dtype=BF16))
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, y, z in graphs:
            for got, want in ((y, formula(q, kp, vp, k, v, n)), (z, formula(q, None, None, k, v, n))):
                assert bool(((got.double() - want[0]).abs() <= want[2]).all())


def test_captured_with_own_keys_beside_the_shared_ones():
    """Enough rows that the shared keys' tiles and the own keys run at the same time; two such calls on two
    streams as well."""
    B, P, L, Hq, Hkv, d = 40, 900, 130, 16, 2, 64
    q, k, v = (normal(i, B, n, h, d, dtype=BF16) for i, n, h in ((1, 1, Hq), (2, L, Hkv), (3, L, Hkv)))
    kp, vp = normal(4, P, Hkv, d, dtype=BF16), normal(5, P, Hkv, d, dtype=BF16)
    n = torch.full((B,), L, dtype=torch.int32, device="cuda")
    lola.prefix_attention(q, kp, vp, k, v, own_len=n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lola.prefix_attention(q, kp, vp, k, v, own_len=n)
    for seed in (7, 8, 9):
        n.copy_(torch.randint(0, L + 1, (B,), generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        q.copy_(normal(seed, *q.shape, dtype=BF16))
        g.replay()
        torch.cuda.synchronize()
        want = formula(q, kp, vp, k, v, n)
        assert bool(((y.double() - want[0]).abs() <= want[2]).all())
    one = lola.prefix_attention(q, kp, vp, k, v, own_len=n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [lola.prefix_attention(q, kp, vp, k, v, own_len=n, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, one) for x in got)


def test_own_scratch_too_small_or_misplaced_is_refused():
    q, k = normal(1, 2, 1, 8, 128, dtype=BF16), normal(2, 2, 5000, 2, 128, dtype=BF16)
    n = lola.attention_workspace(q, k)
    assert n > 0
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(lola.LolaError, match="BUF_TOO_SMALL"):
        lola.cross_attention(q, k, k, workspace=ws[:n - 1])
    with pytest.raises(lola.LolaError, match="256-byte"):
        lola.cross_attention(q, k, k, workspace=ws[16:])
    check(*run_cross(q, k, k, workspace=ws), formula(q, None, None, k, k))


def test_refusals():
    q, k = normal(1, 2, 3, 4, 64, dtype=BF16), normal(2, 2, 9, 2, 64, dtype=BF16)
    f = lola.cross_attention
    for bad in (dict(q=q.float()), dict(v=k[:, :8]), dict(k=k.float()), dict(q=q.cpu()), dict(q=q.half()),
                dict(kv_len=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(kv_len=ints(1, 2, 3)),
                dict(y=torch.empty(2, 3, 4, 64, device="cuda")), dict(lse=torch.empty(2, 3, device="cuda")),
                dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(workspace=torch.empty(8, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f(**{**dict(q=q, k=k, v=k), **bad})
    for bad, text in ((dict(q=q[:, :, :3]), "heads"), (dict(scale=0.0), "scale"), (dict(scale=math.nan), "scale"),
                      (dict(k=k[:, :1].expand(-1, 9, -1, -1)), "stride")):
        with pytest.raises(lola.LolaError, match=text):
            f(**{**dict(q=q, k=k, v=k), **bad})
    wide = torch.zeros(2, 9, 2, 68, dtype=BF16, device="cuda")
    with pytest.raises(lola.LolaError, match="stride"):
        f(q, wide[..., :64], k)
    with pytest.raises(lola.LolaError, match="aligned"):
        f(q, torch.zeros(2 * 9 * 2 * 64 + 8, dtype=BF16, device="cuda")[4:4 + 2 * 9 * 2 * 64].view(2, 9, 2, 64), k)
    with pytest.raises(lola.LolaError, match="d="):
        f(q[..., :32].contiguous(), k[..., :32].contiguous(), k[..., :32].contiguous())
    with pytest.raises((TypeError, ValueError)):
        lola.prefix_attention(q, k, k, k, k)
    with pytest.raises((TypeError, ValueError)):
        lola.prefix_attention(q, None, None, k, k)
