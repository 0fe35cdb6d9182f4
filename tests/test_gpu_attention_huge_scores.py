"""Finite scores far beyond those of any model (scale q.k from 10^6 to 10^11): a row reads its largest
key and nothing else.

q is a power of two times a row of signs, keys are whole multiples of the same signs: every score is exact
in f32 whatever the order of its sum, a row's largest is its only one, and the next differs by more than
10^5.  So p is 1 there (and 0 elsewhere, to 64 bits too), y is that key's value exactly, and lse = scale
q.k there, off by the rounding of scale log2(e) (twice), of its product, of ln 2 and of the last product:
5 x 2^-24 of it."""
import math

import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_attention import BF16, F32, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,S", [(1, 40), (3, 300), (150, 40), (300, 700)])
@pytest.mark.parametrize("scale", [0.125, 0.3, 0.09])
@pytest.mark.parametrize("low,high", [(1, 256), (3, 253)])
def test_the_largest_key_is_read(dtype, T, S, scale, low, high):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    B, H, d = 2, 2, 64
    g = torch.Generator("cuda").manual_seed(T * S)
    signs = torch.randint(0, 2, (d,), generator=g, device="cuda") * 2.0 - 1
    weight = torch.stack([torch.randperm(S, generator=g, device="cuda") for _ in range(B * H)]).view(B, H, S)
    # `low` and `high` once each, the others between them
    weight = torch.where(weight < 2, low + (high - low) * weight, low + 1 + weight % (high - low - 2))
    k = (weight.transpose(1, 2).double()[..., None] * 2.0**9 * signs).to(dtype)
    rows = 2.0 ** torch.randint(11, 16, (B, T, H, 1), generator=g, device="cuda")
    q = (rows * (torch.randint(0, 2, (B, T, H, 1), generator=g, device="cuda") * 2 - 1) * signs).to(dtype)
    v = normal(3, B, S, H, d, dtype=dtype)
    x = torch.einsum("bthd,bshd->bths", q.double(), k.double()) * scale
    top, at = x.max(-1, keepdim=True)
    assert float(top.abs().min()) > 1e6 and float((top - x)[x != top].min()) > 1e5
    want = v.transpose(1, 2)[torch.arange(B, device="cuda")[:, None, None], torch.arange(H, device="cuda"), at[..., 0]]
    lse = torch.full((B, T, H), math.nan, device="cuda")
    y = torch.full_like(q, math.nan)
    lola.cross_attention(q, k, v, scale=scale, y=y, lse=lse)
    assert torch.equal(y, want)
    assert bool(((lse.double() - top[..., 0]).abs() <= 5 * 2.0**-24 * top[..., 0].abs()).all())
