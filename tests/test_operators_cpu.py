"""CPU checks of the fork and attention entry points: what they refuse, before any CUDA call."""
import ctypes

import pytest

import sparse_kv_caching_b200 as lola
from sparse_kv_caching_b200 import build as lbuild

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    lbuild.build()
    return lola.lib()


def config(**kw):
    c = dict(B=2, T=3, Hq=8, Hkv=2, d=64, dtype=lola.DTYPE_BF16, P=0, L=100, scale=0.125)
    c.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    H, d = c["Hkv"], 64
    strides = dict(q_stride=(3 * 8 * d, 8 * d, d), kp_stride=(H * d, d), vp_stride=(H * d, d),
                   k_stride=(100 * H * d, H * d, d), v_stride=(100 * H * d, H * d, d))
    strides.update({k: v for k, v in kw.items() if k.endswith("stride")})
    x = lola.LolaAttnConfig(*c.values())
    for k, v in strides.items():
        setattr(x, k, (ctypes.c_longlong * len(v))(*v))
    return x


@pytest.mark.parametrize("kw,code,text", [
    (dict(B=0), -1, "B=0"), (dict(T=0), -1, "T=0"), (dict(Hq=7), -1, "Hq=7"), (dict(Hkv=0), -1, "Hkv=0"),
    (dict(B=65536), -1, "B=65536"), (dict(B=60000, T=60000), -5, "2^31"), (dict(L=-1), -1, "L=-1"),
    (dict(P=-1), -1, "P=-1"), (dict(d=96), -5, "d=96"), (dict(dtype=2), -1, "dtype=2"), (dict(scale=0.0), -1, "scale"),
    (dict(scale=-1.0), -1, "scale"), (dict(scale=float("inf")), -1, "scale"), (dict(scale=float("nan")), -1, "scale"),
    (dict(q_stride=(1, 64, 64)), -1, "q batch"), (dict(k_stride=(128, 0, 64)), -1, "k token"),
    (dict(v_stride=(128, 128, 4)), -1, "v head"), (dict(k_stride=(-128, 128, 64)), -1, "k batch"),
    (dict(P=5, kp_stride=(0, 64)), -1, "k_prefix token"), (dict(P=5, vp_stride=(128, 3)), -1, "v_prefix head"),
    (dict(dtype=0, q_stride=(8, 8, 2)), -1, "q head"),
])
def test_bad_attention_configs_are_refused(L, kw, code, text):
    n = ctypes.c_size_t()
    assert L.lola_attn_workspace(ctypes.byref(config(**kw)), ctypes.byref(n)) == code
    assert text in L.lola_last_error_string().decode()


def test_strides_that_are_never_used_are_not_looked_at(L):
    n = ctypes.c_size_t()
    for kw in (dict(B=1, q_stride=(3, 512, 64), k_stride=(1, 128, 64)), dict(T=1, q_stride=(512, 5, 64)),
               dict(L=1, k_stride=(128, 7, 64)), dict(L=0, k_stride=(1, 1, 1)), dict(kp_stride=(1, 1))):
        assert L.lola_attn_workspace(ctypes.byref(config(**kw)), ctypes.byref(n)) == 0, kw


def test_attention_arguments_are_refused(L):
    buf = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(buf) + 255) & ~255
    ok, odd, none = VP(p), VP(p + 8), VP(None)
    c, cp = ctypes.byref(config()), ctypes.byref(config(P=7))

    def cross(cfg=c, q=ok, k=ok, v=ok, n=none, y=ok, lse=none, ws=none, size=0):
        return L.lola_cross_attention(cfg, q, k, v, n, y, lse, ws, size, none)

    def prefix(cfg=cp, q=ok, kp=ok, vp=ok, k=ok, v=ok, n=none, y=ok, lse=none, ws=none, size=0):
        return L.lola_prefix_attention(cfg, q, kp, vp, k, v, n, y, lse, ws, size, none)

    for kw in (dict(cfg=None), dict(q=none), dict(k=none), dict(v=none), dict(y=none), dict(q=odd), dict(k=odd),
               dict(v=odd), dict(y=odd), dict(n=VP(p + 2)), dict(lse=VP(p + 1)), dict(cfg=cp)):
        assert cross(**kw) == -1, kw
    for kw in (dict(cfg=None), dict(kp=none), dict(vp=none), dict(kp=odd), dict(vp=odd), dict(k=none), dict(y=none)):
        assert prefix(**kw) == -1, kw
    assert L.lola_attn_workspace(c, None) == -1


def test_fork_arguments_are_refused(L):
    assert L.lola_state_fork(None, None, None, 1, None) == -1
    assert L.lola_set_batch(None, 1) == -1
