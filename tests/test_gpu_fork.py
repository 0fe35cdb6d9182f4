"""Forks of whole sequences (lola_state_fork, lola_set_batch): the copied memories bit for bit, and
that the layer goes on as if each sequence had been processed by itself."""
import random

import numpy as np
import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests import parity as P

pytestmark = pytest.mark.gpu
MEMORIES = ("H", "s", "cache_k", "cache_v", "cache_phik", "cache_pos", "win_k", "win_v", "win_phik")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


SHAPES = [  # Hq, Hkv, d, Dh, eta, lam, dtype: odd sizes end inside 16 bytes (cache_pos)
    (4, 2, 64, 32, 16, 24, "f32"), (3, 1, 128, 64, 7, 13, "bf16"), (8, 8, 64, 64, 33, 0, "bf16"),
    (1, 1, 64, 32, 1, 1, "f32"),
]


def layer(B, shape, T=64, seed=0):
    Hq, Hkv, d, Dh, eta, lam, dtype = shape
    cfg = lola.make_config(B, Hq, Hkv, d, Dh, eta, lam, 16, dtype, T)
    g = torch.Generator("cuda").manual_seed(99)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    return lola.LolaLayer(cfg, (torch.randn(Hkv, d, Dh, generator=g, device="cuda") / d ** 0.5).to(t))


def tokens(lay, T, seed, B=None):
    c, B = lay.cfg, B or lay.B
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(B, T, h, c.d, generator=g, device="cuda").to(lay.dtype) for h in (c.Hq, c.Hkv, c.Hkv)]


def memories(lay):
    e = lay.export()
    return {m: e[m].clone().view(lay.B, lay.cfg.Hkv, *e[m].shape[1:]) for m in MEMORIES}


def step(lay, x, t):
    return lay.decode(*(a[:, t].contiguous() for a in x))


def index(p):
    return torch.tensor(p, dtype=torch.int32, device="cuda")


def assert_forked(lay, before, parents):
    after = memories(lay)
    for m in MEMORIES:
        assert torch.equal(after[m], before[m][torch.tensor(parents, device="cuda").long()]), m


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("B,parents", [(1, [0]), (1, [0] * 37), (5, [4, 4, 0, 2]), (3, [2, 1, 0, 0, 1, 2, 2]),
                                       (20, list(range(19, -1, -1)))])
def test_between_two_layers(shape, B, parents):
    src, dst = layer(B, shape), layer(len(parents) + 1, shape)
    x = tokens(src, 64, 1)
    src.prefill(*x)
    before = memories(src)
    dst.prefill(*tokens(dst, 64, 2))            # what the destination held is gone
    dst.fork(index(parents), src=src)
    assert dst.B == len(parents) and dst.export()["t"] == 64
    assert_forked(dst, before, parents)
    for m, y in memories(src).items():
        assert torch.equal(y, before[m])
    dst.check()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("B,room,parents", [
    (2, 2, [1, 0]), (6, 6, [1, 2, 3, 4, 5, 0]), (6, 6, [0, 1, 2, 3, 4, 5]), (6, 6, [3, 3, 3, 3, 3, 3]),
    (6, 6, [5, 1, 0]), (1, 9, [0] * 9), (4, 40, [i * 7 % 4 for i in range(40)]), (64, 64, None), (150, 150, None),
    (500, 500, None)])
def test_in_place(shape, B, room, parents):
    if parents is None:
        parents = [random.Random(B).randrange(B) for _ in range(B)]
    lay = layer(room, shape, T=32)
    lay.set_batch(B)
    lay.prefill(*tokens(lay, 32, 1))
    before = memories(lay)
    lay.fork(index(parents))
    assert lay.B == len(parents)
    assert_forked(lay, before, parents)
    lay.check()


@pytest.mark.parametrize("scorer", ["sre", "attn"])
@pytest.mark.parametrize("prefill_only", [False, True])
def test_decode_goes_on_after_a_fork(scorer, prefill_only):
    """Forked sequences decode bit for bit like a layer that processed them from the start."""
    shape = (4, 2, 64, 32, 12, 20, "bf16")
    parents = [1, 1, 0, 2, 1]
    a, b = layer(5, shape), layer(5, shape)
    for lay in (a, b):
        lay.set_scorer(scorer)
    x = tokens(a, 48, 1, B=3)
    steps = 0 if prefill_only else 5
    a.set_batch(3)
    a.prefill(*x)
    pick = torch.tensor(parents, device="cuda")
    b.prefill(*(z[pick].contiguous() for z in x))
    d = tokens(a, 5, 2, B=3)
    for t in range(steps):
        step(a, d, t)
        step(b, [z[pick] for z in d], t)
    a.fork(index(parents))
    e = tokens(b, 20, 3)
    for t in range(20):
        assert torch.equal(step(a, e, t), step(b, e, t)), t
    ma, mb = memories(a), memories(b)
    for m in MEMORIES:
        assert torch.equal(ma[m], mb[m]), m
    a.check()


def test_prefill_goes_on_after_a_fork():
    shape = (4, 2, 64, 32, 12, 20, "f32")
    a, b = layer(4, shape), layer(4, shape)
    x = tokens(a, 64, 1, B=1)
    a.set_batch(1)
    a.prefill(*x)
    a.fork(index([0, 0, 0, 0]))
    b.prefill(*(z.expand(4, -1, -1, -1).contiguous() for z in x))
    y = tokens(a, 64, 2)
    ya, yb = a.prefill(*y), b.prefill(*y)
    # (another number of streams may choose another chain kernel: f32 rounding, not bits)
    assert P.max_rel(ya.cpu().numpy(), yb.cpu().numpy()) < P.TOL["f32"]


def test_batch_and_reset():
    lay = layer(4, SHAPES[0])
    lay.set_batch(2)
    assert lay.prefill(*tokens(lay, 16, 1)).shape[0] == 2
    with pytest.raises(lola.LolaError, match="before the first token"):
        lay.set_batch(3)
    with pytest.raises(ValueError):
        lay.prefill(*tokens(lay, 16, 1, B=4))
    lay.fork(index([0, 1, 1]))
    lay.reset()
    assert lay.B == 4 and lay.prefill(*tokens(lay, 16, 1)).shape[0] == 4
    full = layer(4, SHAPES[0])
    full.prefill(*tokens(full, 16, 1))
    for m, x in memories(full).items():
        assert torch.equal(x, memories(lay)[m])


def test_a_parent_outside_is_reported_and_nothing_else_changes():
    lay, dst = layer(3, SHAPES[0]), layer(3, SHAPES[0])
    lay.prefill(*tokens(lay, 64, 1))
    before = memories(lay)
    lay.fork(index([2, 3, -1]))
    with pytest.raises(lola.LolaError, match="INVALID_ARG"):
        lay.check()
    assert_forked(lay, before, [2, 1, 2])
    lay.reset()
    lay.check()
    lay.set_batch(2)
    lay.prefill(*tokens(lay, 64, 1))
    dst.fork(index([0, 2]), src=lay)             # only two sequences are live
    with pytest.raises(lola.LolaError, match="INVALID_ARG"):
        dst.check()


def test_sre_map_needs_a_new_prefill():
    lay = layer(2, SHAPES[0])
    x = tokens(lay, 64, 1)
    lay.prefill(*x)
    lay.fork(index([1, 0]))
    with pytest.raises(lola.LolaError, match="prefill"):
        lay.sre_map(x[1], x[2])


def test_captured_and_replayed_with_other_parents():
    src, dst = layer(4, SHAPES[1]), layer(3, SHAPES[1])
    src.prefill(*tokens(src, 64, 1))
    before = memories(src)
    p = index([0, 0, 0])
    dst.fork(p, src=src)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dst.fork(p, src=src)
    for parents in ([3, 1, 1], [2, 0, 3]):
        p.copy_(index(parents))
        g.replay()
        torch.cuda.synchronize()
        assert_forked(dst, before, parents)


def test_side_stream():
    src, dst = layer(2, SHAPES[1]), layer(8, SHAPES[1])
    src.prefill(*tokens(src, 64, 1))
    before = memories(src)
    p = index([1, 0] * 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    dst.fork(p, src=src, stream=side)
    side.synchronize()
    assert_forked(dst, before, [1, 0] * 4)


def test_refusals():
    a = layer(2, SHAPES[0])
    for bad in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32),
                torch.zeros(4, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            a.fork(bad)
    with pytest.raises(TypeError):
        a.fork([0, 1])
    with pytest.raises(lola.LolaError, match="INVALID_ARG"):
        a.fork(index([0, 1, 0]))                 # more than the layer holds
    with pytest.raises(lola.LolaError, match="INVALID_ARG"):
        a.fork(index([]))
    with pytest.raises(lola.LolaError, match="differ"):
        a.fork(index([0]), src=layer(2, (4, 2, 64, 32, 16, 25, "f32")))
    assert a.B == 2
    np.testing.assert_equal(a.export()["t"], 0)
