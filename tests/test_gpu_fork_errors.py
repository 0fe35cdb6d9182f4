"""A fork with a bad parent: what lola_state_check asks for is what helps."""
import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_fork import SHAPES, assert_forked, index, layer, memories, tokens

pytestmark = pytest.mark.gpu


def test_reset_then_fork_again():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    src, dst = layer(2, SHAPES[0]), layer(3, SHAPES[0])
    src.prefill(*tokens(src, 64, 1))
    before = memories(src)
    dst.fork(index([0, 2, 1]), src=src)                # sequence 2 does not exist
    with pytest.raises(lola.LolaError, match="INVALID_ARG.*reset the state, then fork again"):
        dst.check()
    dst.fork(index([0, 1, 1]), src=src)                # a good fork alone does not clear it
    with pytest.raises(lola.LolaError, match="INVALID_ARG"):
        dst.check()
    dst.reset()
    dst.check()
    dst.fork(index([0, 1, 1]), src=src)
    dst.check()
    assert_forked(dst, before, [0, 1, 1])
