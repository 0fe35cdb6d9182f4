"""Every element of y and lse is written by the call: both start as NaN.  The cases of
test_gpu_attention.py, and keys that the whole batch shares and that are its only ones (one encoder
output for all sequences, a prefix with no keys behind it) on both sides of the 16 query rows per kv head
and the 512 shared keys at which the work is cut another way.  Tolerances: see test_gpu_attention.py."""
import math

import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_attention import BF16, CROSS, F32, PREFIX, check, formula, ints, normal

pytestmark = pytest.mark.gpu
TYPES = [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    lola.attention_check()


def unwritten(q):
    return (torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda"),
            torch.full(q.shape[:3], math.nan, device="cuda"))


def cross(q, k, v, n=None, **kw):
    y, lse = unwritten(q)
    return lola.cross_attention(q, k, v, kv_len=n, y=y, lse=lse, **kw), lse


def prefix(q, kp, vp, k, v, n=None, **kw):
    y, lse = unwritten(q)
    return lola.prefix_attention(q, kp, vp, k, v, own_len=n, y=y, lse=lse, **kw), lse


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("B,T,S,Hq,Hkv,lens", CROSS)
def test_cross(dtype, d, B, T, S, Hq, Hkv, lens):
    q, k, v = normal(1, B, T, Hq, d, dtype=dtype), normal(2, B, S, Hkv, d, dtype=dtype), normal(3, B, S, Hkv, d, dtype=dtype)
    n = None if lens is None else ints(*lens)
    check(*cross(q, k, v, n), formula(q, None, None, k, v, n))


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("B,T,P,L,Hq,Hkv,lens", PREFIX)
def test_prefix(dtype, d, B, T, P, L, Hq, Hkv, lens):
    q = normal(1, B, T, Hq, d, dtype=dtype)
    kp, vp = normal(2, P, Hkv, d, dtype=dtype), normal(3, P, Hkv, d, dtype=dtype)
    k, v = normal(4, B, L, Hkv, d, dtype=dtype), normal(5, B, L, Hkv, d, dtype=dtype)
    n = None if lens is None else ints(*lens)
    check(*prefix(q, kp, vp, k, v, n), formula(q, kp, vp, k, v, n))


SHARED = [  # B, T, keys, Hq, Hkv; query rows per kv head: B T Hq / Hkv
    (5, 1, 1500, 20, 20), (2, 1, 1500, 32, 8), (4, 1, 1500, 32, 8), (5, 1, 1500, 32, 8),
    (2, 4, 4096, 16, 8), (16, 1, 513, 8, 8), (17, 1, 513, 8, 8), (3, 1, 513, 1, 1), (3, 1, 512, 1, 1),
    (2, 1, 4096, 1, 1), (8, 2, 4096, 1, 1), (2, 2, 600, 20, 20), (2, 1, 577, 300, 300), (2, 40, 700, 4, 2),
]


@pytest.mark.parametrize("dtype,d", TYPES)
@pytest.mark.parametrize("B,T,N,Hq,Hkv", SHARED)
def test_keys_that_the_batch_shares_alone(dtype, d, B, T, N, Hq, Hkv):
    q, k, v = (normal(i, *s, d, dtype=dtype) for i, s in ((1, (B, T, Hq)), (2, (N, Hkv)), (3, (N, Hkv))))
    none = torch.empty(B, 0, Hkv, d, dtype=dtype, device="cuda")
    kb, vb = k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1)
    want = formula(q, None, None, kb, vb)
    check(*cross(q, kb, vb), want)                     # one encoder output, no lengths
    check(*prefix(q, k, v, none, none), want)          # a prefix and nothing else
    few = ints(*[(b * 977) % (N + 1) for b in range(B)])
    check(*cross(q, kb, vb, few), formula(q, None, None, kb, vb, few))


@pytest.mark.parametrize("B,T,N,Hq,Hkv", [(5, 1, 1500, 20, 20), (2, 4, 4096, 16, 8)])
def test_shared_keys_alone_captured_and_replayed(B, T, N, Hq, Hkv):
    q, k, v = (normal(i, *s, 64, dtype=BF16) for i, s in ((1, (B, T, Hq)), (2, (N, Hkv)), (3, (N, Hkv))))
    kb, vb = k.expand(B, -1, -1, -1), v.expand(B, -1, -1, -1)
    y, lse = unwritten(q)
    lola.cross_attention(q, kb, vb)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lola.cross_attention(q, kb, vb, y=y, lse=lse)
    for seed in (7, 8):
        q.copy_(normal(seed, *q.shape, dtype=BF16))
        y.fill_(math.nan)
        lse.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        check(y, lse, formula(q, None, None, kb, vb))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,G", [(2, 4), (6, 3), (200, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_keys_behind_the_own_position_do_not_matter(dtype, T, G, bad):
    """NaN and infinities in the key of each sequence's last token: every query but the last is as without."""
    B, L, Hkv, d = 3, 333, 2, 128
    q, k, v = normal(1, B, T, G * Hkv, d, dtype=dtype), normal(2, B, L, Hkv, d, dtype=dtype), normal(3, B, L, Hkv, d, dtype=dtype)
    kp, vp = normal(4, 600, Hkv, d, dtype=dtype), normal(5, 600, Hkv, d, dtype=dtype)
    n = ints(333, 230, 205)
    want = formula(q, kp, vp, k, v, n)
    for b in range(B):
        k[b, int(n[b]) - 1] = bad
    y, lse = prefix(q, kp, vp, k, v, n)
    check(y[:, :-1], lse[:, :-1], tuple(x[:, :-1] for x in want))
