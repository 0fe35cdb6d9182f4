"""Forks in place from several host threads, each with a layer and a stream of its own."""
import ctypes
import threading

import pytest
import torch

import sparse_kv_caching_b200 as lola
from tests.test_gpu_fork import assert_forked, index, layer, memories, tokens

pytestmark = pytest.mark.gpu
SHAPE = (1, 1, 64, 32, 1, 1, "f32")


def test_forks_of_different_sizes_at_the_same_time():
    """A launch asks for the shared memory of its own number of sequences: another thread's fork of fewer
    may not lower what this one is allowed.  The C calls themselves, one behind the other, so that the
    threads meet inside them (a third of the largest failed so)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    work = []
    for i, n in enumerate((1500, 1400, 5, 60)):
        lay = layer(n, SHAPE, T=16)
        lay.prefill(*tokens(lay, 16, i))
        work.append((lay, memories(lay), index(list(range(n))), torch.cuda.Stream()))
    torch.cuda.synchronize()
    call, times, failed = lola.lib().lola_state_fork, 3000, []
    begin = threading.Barrier(len(work))

    def forks(lay, parents, stream):
        args = (lay.handle, lay.handle, ctypes.c_void_p(parents.data_ptr()), parents.numel(),
                ctypes.c_void_p(stream.cuda_stream))
        begin.wait()
        bad = sum(call(*args) != 0 for _ in range(times))
        if bad:
            failed.append((parents.numel(), bad))

    threads = [threading.Thread(target=forks, args=(lay, p, s)) for lay, _, p, s in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for lay, before, p, s in work:
        n = p.numel()
        turn = [(b + 1) % n for b in range(n)]        # every sequence moves and is a parent of another
        lay.fork(index(turn))
        torch.cuda.synchronize()
        assert_forked(lay, before, turn)
        lay.check()
