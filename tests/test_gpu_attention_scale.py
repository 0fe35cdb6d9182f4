"""scale as a 0-d tensor: every call takes the value that it has at that call."""
import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_attention import BF16, F32, formula, check, normal, run_cross, run_prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("device", ["cpu", "cuda"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_that_changes_in_place(dtype, device):
    q, k, v = (normal(i, 2, n, 4, 64, dtype=dtype) for i, n in ((1, 3), (2, 150), (3, 150)))
    scale = torch.tensor(0.125, device=device)
    for value in (0.125, 0.5, 0.25):
        scale.fill_(value)
        check(*run_cross(q, k, v, scale=scale), formula(q, None, None, k, v, scale=value))
        check(*run_prefix(q, k[0], v[0], k, v, scale=scale), formula(q, k[0], v[0], k, v, scale=value))
