"""The decoder of test_gpu_together.py with every exact attention call checked as it happens, element by
element, against the formula in 64 bits on the very tensors that the call was given (tolerances: see
test_gpu_attention.py), and the hybrid layer's forked memories bit for bit: samples of one prompt, a shared
prefix, one encoder output for all, a beam step, a smaller batch."""
import math

import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_attention import check, formula
from tests.test_gpu_fork import MEMORIES, memories
from tests.test_gpu_together import PROMPT, STEPS, WIDTH, Decoder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [3, 20])
def test_each_call_of_a_decoder(monkeypatch, N):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    calls, cross, prefix = [], lola.cross_attention, lola.prefix_attention

    def unwritten(q):
        return dict(y=torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda"),
                    lse=torch.full(q.shape[:3], math.nan, device="cuda"))

    def checked_cross(q, k, v):
        out = unwritten(q)
        cross(q, k, v, **out)
        check(out["y"], out["lse"], formula(q, None, None, k, v))
        calls.append("cross")
        return out["y"]

    def checked_prefix(q, kp, vp, k, v, own_len=None):
        out = unwritten(q)
        prefix(q, kp, vp, k, v, own_len=own_len, **out)
        check(out["y"], out["lse"], formula(q, kp, vp, k, v, own_len))
        calls.append("prefix")
        return out["y"]

    monkeypatch.setattr(lola, "cross_attention", checked_cross)
    monkeypatch.setattr(lola, "prefix_attention", checked_prefix)
    g = torch.Generator("cuda").manual_seed(1)
    prompt = torch.randn(1, PROMPT, WIDTH, generator=g, device="cuda").bfloat16()
    a = Decoder(N)
    a.layer.set_batch(1)
    x = a.prompt(prompt, True)[:, -1:].expand(N, -1, -1)
    forks = {0: [0] * N, 4: [i * 7 % N for i in range(N)], 8: [N - 1, N - 1, 0]}
    for t in range(STEPS):
        if t in forks:
            p = torch.tensor(forks[t], dtype=torch.int32, device="cuda")
            before, own = memories(a.layer), [z.clone() for z in a.own]
            a.fork(p)
            after = memories(a.layer)
            assert all(torch.equal(after[m], before[m][p.long()]) for m in MEMORIES)
            assert all(torch.equal(z, w[p.long()]) for z, w in zip(a.own, own))
            x = x[p.long()]
        x = a.step(x + torch.randn(x.shape, generator=g, device="cuda").bfloat16())
        assert torch.isfinite(x.double()).all()
    assert x.shape[0] == 3 and calls == ["prefix", "cross"] * (STEPS + 1)
    a.layer.check()
    lola.attention_check()
