"""Layers of different sizes used from several host threads at the same time, each on a stream of its own."""
import ctypes
import threading

import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_fork import layer, memories, tokens

pytestmark = pytest.mark.gpu
SIZES = [(200, 300), (3, 2), (40, 64), (7, 150)]      # eta, lambda: the kernels' shared memory grows with them


def shape(eta, lam, dtype):
    return (2, 1, 64, 32, eta, lam, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what,times", [("decode", 3000), ("prefill", 1000)])
def test_calls_of_different_sizes_at_the_same_time(dtype, what, times):
    """A launch asks for the shared memory of its own layer: another thread's smaller layer may not lower
    what this one is allowed.  Afterwards each layer holds what it holds when it is used alone."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    T = 1 if what == "decode" else 16

    def made():
        out = []
        for i, (eta, lam) in enumerate(SIZES):
            lay = layer(1, shape(eta, lam, dtype), T=16)
            x = [z[:, :T].contiguous() for z in tokens(lay, 16, i)]
            y = torch.empty(x[0].shape, dtype=torch.float32, device="cuda")
            out.append((lay, x, y, torch.cuda.Stream()))
        torch.cuda.synchronize()
        return out

    L = lola.lib()

    def calls(lay, x, y, stream):
        p = [ctypes.c_void_p(z.data_ptr()) for z in x]
        s = ctypes.c_void_p(stream.cuda_stream)
        if what == "decode":
            one = lambda: L.lola_decode_step(lay.handle, *p, ctypes.c_void_p(y.data_ptr()), s)
        else:
            one = lambda: L.lola_prefill_chunked(lay.handle, *p, 16, ctypes.c_void_p(y.data_ptr()), s)
        return sum(one() != 0 for _ in range(times))

    alone = made()
    for w in alone:
        assert calls(*w) == 0
    torch.cuda.synchronize()
    together, failed = made(), []
    begin = threading.Barrier(len(together))

    def run(w):
        begin.wait()
        bad = calls(*w)
        if bad:
            failed.append((w[0].cfg.lambda_, bad))

    threads = [threading.Thread(target=run, args=(w,)) for w in together]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (a, _, ya, _), (b, _, yb, _) in zip(alone, together):
        assert torch.equal(ya, yb)
        ma, mb = memories(a), memories(b)
        assert all(torch.equal(ma[m], mb[m]) for m in ma)
        b.check()
