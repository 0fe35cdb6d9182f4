"""CPU checks of what the attention binding hands on."""
import pytest
import torch

import sparse_kv_caching_b200 as lola


class Planned(BaseException):
    pass


def test_scale_is_read_at_every_call(monkeypatch):
    """The plan of a call is looked up by values: a tensor would be looked up by its identity and keep
    the value it had at first."""
    seen = []

    def plan(*key):
        seen.append(key[-1])
        raise Planned

    monkeypatch.setattr(lola, "_attn_plan", plan)
    x = torch.zeros(1, 1, 1, 64)
    scale = torch.tensor(0.125)
    for value in (0.125, 0.5):
        scale.fill_(value)
        with pytest.raises(Planned):
            lola.cross_attention(x, x, x, scale=scale)
        with pytest.raises(Planned):
            lola.prefix_attention(x, x[0], x[0], x, x, scale=scale)
    with pytest.raises(Planned):
        lola.cross_attention(x, x, x)
    assert all(type(s) is float for s in seen[:4])
    assert seen == [0.125, 0.125, 0.5, 0.5, None]


@pytest.mark.parametrize("scale", ["1", torch.zeros(2), 1j])
def test_scale_that_is_no_number_is_refused(monkeypatch, scale):
    def plan(*key):
        raise Planned

    monkeypatch.setattr(lola, "_attn_plan", plan)
    x = torch.zeros(1, 1, 1, 64)
    with pytest.raises((TypeError, ValueError, RuntimeError)) as e:
        lola.cross_attention(x, x, x, scale=scale)
