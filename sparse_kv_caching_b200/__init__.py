"""B200 (sm_100a) LoLA hybrid-attention layer: Python binding of include/lola.h.

The binding only marshals arguments: it checks dtypes, shapes and devices of
torch tensors, passes their device pointers and the current CUDA stream to
the C ABI of liblola.so, and wraps device views of the state.  Every step of
the layer runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or fails to load, every entry point raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, byref, c_float, c_int, c_longlong, c_size_t, c_void_p, c_char_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblola.so")

DTYPE_F32, DTYPE_BF16 = 0, 1
_TORCH_DTYPE = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16}
_DTYPE_CODE = {t: c for c, t in _TORCH_DTYPE.items()}
ERRORS = {0: "OK", -1: "INVALID_ARG", -2: "BUF_TOO_SMALL", -3: "CUDA", -4: "TIMEOUT", -5: "UNSUPPORTED"}

# Every entry point of include/lola.h.
EXPORTS = ("lola_state_bytes", "lola_state_init", "lola_state_reset", "lola_state_free",
           "lola_prefill_chunked", "lola_decode_step", "lola_prefill_chunked_host",
           "lola_decode_step_host", "lola_state_export", "lola_profile_enable",
           "lola_profile_read", "lola_launch_count", "lola_prefill_once_noalloc", "lola_selftest_umma",
           "lola_set_read_options", "lola_sre_map", "lola_set_scorer", "lola_state_check",
           "lola_set_batch", "lola_state_fork", "lola_attn_workspace", "lola_cross_attention",
           "lola_prefix_attention", "lola_attn_check",
           "lola_last_error_string")
KERNEL_CLASSES = ("phi", "scan", "output", "finalize", "decode", "sre_map", "scores")
READ_HIDE_STATE, READ_HIDE_SPARSE = 1, 2
SCORERS = ("sre", "kernel_sq", "kernel_abs", "kernel_ratio", "attn")   # LOLA_SCORE_* in this order


class LolaConfig(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hq", c_int), ("Hkv", c_int), ("d", c_int), ("Dh", c_int),
                ("eta", c_int), ("lambda_", c_int), ("chunk", c_int), ("dtype", c_int),
                ("max_tokens", c_int)]


class LolaStateView(ctypes.Structure):
    _fields_ = [("t", c_longlong), ("n_cache", c_int), ("H", c_void_p), ("s", c_void_p),
                ("cache_k", c_void_p), ("cache_v", c_void_p), ("cache_phik", c_void_p),
                ("cache_pos", c_void_p), ("win_k", c_void_p), ("win_v", c_void_p),
                ("win_phik", c_void_p), ("trace_pos", c_void_p), ("trace_len", c_int),
                ("trace_stride", c_int), ("trace_t0", c_longlong), ("err_word", c_void_p)]


class LolaAttnConfig(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("Hq", c_int), ("Hkv", c_int), ("d", c_int), ("dtype", c_int),
                ("P", c_int), ("L", c_int), ("scale", c_float), ("q_stride", c_longlong * 3),
                ("kp_stride", c_longlong * 2), ("vp_stride", c_longlong * 2), ("k_stride", c_longlong * 3),
                ("v_stride", c_longlong * 3)]


class LolaError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """Load liblola.so (raises if it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise LolaError(f"{LIB_PATH} is missing; build it with `python -m sparse_kv_caching_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp = c_void_p
    L.lola_state_bytes.argtypes = [POINTER(LolaConfig), POINTER(c_size_t)]
    L.lola_state_init.argtypes = [POINTER(LolaConfig), vp, vp, c_size_t, vp, POINTER(vp)]
    L.lola_state_reset.argtypes = [vp, vp]
    L.lola_state_free.argtypes = [vp]
    L.lola_prefill_chunked.argtypes = [vp, vp, vp, vp, c_int, vp, vp]
    L.lola_decode_step.argtypes = [vp, vp, vp, vp, vp, vp]
    L.lola_prefill_chunked_host.argtypes = [vp, vp, vp, vp, c_int, vp, vp]
    L.lola_decode_step_host.argtypes = [vp, vp, vp, vp, vp, vp]
    L.lola_state_export.argtypes = [vp, POINTER(LolaStateView)]
    L.lola_profile_enable.argtypes = [vp, c_int]
    L.lola_profile_read.argtypes = [vp, POINTER(ctypes.c_float), POINTER(c_longlong), c_int]
    L.lola_prefill_once_noalloc.argtypes = [POINTER(LolaConfig), vp, vp, vp, vp, c_int, vp, vp]
    L.lola_selftest_umma.argtypes = [c_int, vp, vp, vp, c_int, c_int, c_int, vp, vp]
    L.lola_set_read_options.argtypes = [vp, c_int, c_int]
    L.lola_sre_map.argtypes = [vp, vp, vp, c_int, vp, vp, vp]
    L.lola_set_scorer.argtypes = [vp, c_int]
    L.lola_state_check.argtypes = [vp, vp]
    L.lola_set_batch.argtypes = [vp, c_int]
    L.lola_state_fork.argtypes = [vp, vp, vp, c_int, vp]
    L.lola_attn_workspace.argtypes = [POINTER(LolaAttnConfig), POINTER(c_size_t)]
    L.lola_cross_attention.argtypes = [POINTER(LolaAttnConfig), vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
    L.lola_prefix_attention.argtypes = [POINTER(LolaAttnConfig), vp, vp, vp, vp, vp, vp, vp, vp, vp, c_size_t, vp]
    L.lola_attn_check.argtypes = [vp]
    L.lola_launch_count.argtypes = []
    L.lola_launch_count.restype = c_longlong
    L.lola_last_error_string.argtypes = []
    L.lola_last_error_string.restype = c_char_p
    for name in EXPORTS:
        if name not in ("lola_launch_count", "lola_last_error_string"):
            getattr(L, name).restype = c_int
    _lib = L
    return L


def _check(rc: int) -> None:
    if rc != 0:
        msg = lib().lola_last_error_string().decode()
        raise LolaError(f"LOLA_ERR_{ERRORS.get(rc, rc)}: {msg}")


def make_config(B, Hq, Hkv, d, Dh, eta, lam, chunk, dtype, max_tokens) -> LolaConfig:
    dt = {"f32": DTYPE_F32, "bf16": DTYPE_BF16}.get(dtype, dtype)
    return LolaConfig(B, Hq, Hkv, d, Dh, eta, lam, chunk, dt, max_tokens)


def state_bytes(cfg: LolaConfig) -> int:
    n = c_size_t()
    _check(lib().lola_state_bytes(byref(cfg), byref(n)))
    return n.value


def launch_count() -> int:
    """Kernels launched by liblola.so in this process."""
    return int(lib().lola_launch_count())


def prefill_once_noalloc(cfg: LolaConfig, W, q, k, v, y, stream=None):
    """One-shot prefill from an empty state using the library's built-in scratch array.

    For callers that cannot allocate device memory: nothing is allocated here
    or in the library; q, k, v, W and y are the caller's device tensors.
    Calls share the built-in array, so overlapping calls race.
    """
    for x in (W, q, k, v, y):
        if not (isinstance(x, torch.Tensor) and x.is_cuda and x.is_contiguous()):
            raise ValueError("W, q, k, v, y must be contiguous CUDA tensors")
    if y.dtype != torch.float32:
        raise ValueError("y must be float32")
    _check(lib().lola_prefill_once_noalloc(byref(cfg), c_void_p(W.data_ptr()), c_void_p(q.data_ptr()),
                                           c_void_p(k.data_ptr()), c_void_p(v.data_ptr()), q.shape[1],
                                           c_void_p(y.data_ptr()), _stream(stream)))
    return y


# The current stream's handle by device index, without the wrapper object (1 us less a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream=None) -> c_void_p:
    return c_void_p(_raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream)


# -- exact attention beside the layer ---------------------------------------------
def _what(x):
    """What a call's checks and plan depend on: equal for equal shapes, strides, dtypes and devices."""
    return x.shape, x.stride(), x.dtype, x.device


def _attn_same(got, name, shape, dtype, device, packed=False):
    if got[0] != shape:
        raise ValueError(f"{name}: shape {tuple(got[0])}, expected {tuple(shape)}")
    if got[2] != dtype:
        raise ValueError(f"{name}: dtype {got[2]}, expected {dtype}")
    if got[3] != device:
        raise ValueError(f"{name}: on {got[3]}, expected {device}")
    if packed:
        want = 1
        for n, st in zip(reversed(got[0]), reversed(got[1])):
            if n > 1 and st != want:
                raise ValueError(f"{name} must be contiguous")
            want *= n


@functools.lru_cache(maxsize=4096)
def _attn_plan(q, k, v, kp, vp, lens, lens_name, y, lse, scale):
    """(config, bytes of workspace) of a call, from what its tensors are (see _what) alone."""
    qs, q_st, dtype, dev = q
    ks, k_st = k[:2]
    if dev.type != "cuda":
        raise ValueError(f"q: on {dev}, expected a CUDA device")
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"q: dtype {dtype}, expected one of {list(_DTYPE_CODE)}")
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError(f"q and k must have 4 dimensions: shapes {tuple(qs)}, {tuple(ks)}")
    B, T, Hq, d = qs
    L, Hkv = ks[1], ks[2]
    _attn_same(k, "k", (B, L, Hkv, d), dtype, dev)
    _attn_same(v, "v", ks, dtype, dev)
    P = 0
    if kp is not None:
        if len(kp[0]) != 3:
            raise ValueError(f"k_prefix must have 3 dimensions: shape {tuple(kp[0])}")
        P = kp[0][0]
        _attn_same(kp, "k_prefix", (P, Hkv, d), dtype, dev)
        _attn_same(vp, "v_prefix", kp[0], dtype, dev)
    if lens is not None:
        _attn_same(lens, lens_name, (B,), torch.int32, dev, packed=True)
    if y is not None:
        _attn_same(y, "y", qs, dtype, dev, packed=True)
    if lse is not None:
        _attn_same(lse, "lse", qs[:3], torch.float32, dev, packed=True)
    for x, name, n in ((q, "q", B * T * Hq), (k, "k", L), (v, "v", L), (kp, "k_prefix", P), (vp, "v_prefix", P)):
        if n and x[1][-1] != 1:
            raise ValueError(f"{name}: the head's elements must be contiguous (last stride 1)")
    c = LolaAttnConfig(B, T, Hq, Hkv, d, _DTYPE_CODE[dtype], P, L, d ** -0.5 if scale is None else scale, q_st[:3],
                       kp[1][:2] if P else (0, 0), vp[1][:2] if P else (0, 0), k_st[:3], v[1][:3])
    n = c_size_t()
    _check(lib().lola_attn_workspace(byref(c), byref(n)))
    return c, n.value


def _attention(q, kp, vp, k, v, lens, lens_name, scale, y, lse, workspace, stream):
    if scale is not None:
        scale = c_float(scale).value    # the plan is looked up by this value (a tensor would be by its identity)
    try:
        cfg, need = _attn_plan(_what(q), _what(k), _what(v), None if kp is None else _what(kp),
                               None if vp is None else _what(vp), None if lens is None else _what(lens), lens_name,
                               None if y is None else _what(y), None if lse is None else _what(lse), scale)
    except AttributeError:
        for x, name in ((q, "q"), (k, "k"), (v, "v"), (kp, "k_prefix"), (vp, "v_prefix"), (lens, lens_name), (y, "y"),
                        (lse, "lse")):
            if not isinstance(x, torch.Tensor) and (x is not None or name in ("q", "k", "v")):
                raise TypeError(f"{name} must be a torch.Tensor") from None
        raise
    dev = q.device
    if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8
                                      and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream: on {stream.device}, expected {dev}")
    if stream is not None or torch.cuda.current_device() != dev.index:
        # on the tensors' device and the call's stream, so that the allocator orders the reuse
        # of what is allocated here behind the call
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return _attn_call(cfg, need, q, kp, vp, k, v, lens, y, lse, workspace)
    return _attn_call(cfg, need, q, kp, vp, k, v, lens, y, lse, workspace)


def _attn_call(cfg, need, q, kp, vp, k, v, lens, y, lse, workspace):
    if y is None:                                     # (empty_like is the quickest, but keeps q's strides)
        y = torch.empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)
    if workspace is None and need:
        workspace = q.new_empty(-(-need // q.element_size()))
    ws, size = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    n, ls = 0 if lens is None else lens.data_ptr(), 0 if lse is None else lse.data_ptr()
    st = _raw_stream(q.device.index)
    if kp is None:
        rc = _lib.lola_cross_attention(byref(cfg), q.data_ptr(), k.data_ptr(), v.data_ptr(), n, y.data_ptr(), ls, ws,
                                       size, st)
    else:
        rc = _lib.lola_prefix_attention(byref(cfg), q.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.data_ptr(),
                                        v.data_ptr(), n, y.data_ptr(), ls, ws, size, st)
    if rc:
        _check(rc)
    return y


def attention_workspace(q, k, k_prefix=None) -> int:
    """Bytes of scratch that cross_attention(q, k, ...) or prefix_attention(q, k_prefix, ..., k, ...) uses."""
    pre = None if k_prefix is None else _what(k_prefix)
    return _attn_plan(_what(q), _what(k), _what(k), pre, pre, None, "", None, None, 1.0)[1]


def attention_check(stream=None) -> None:
    """Sync point: wait for the stream and raise LolaError (LOLA_ERR_TIMEOUT) if a bounded device-side
    wait of an attention call on the current device gave up since the last check."""
    _check(lib().lola_attn_check(_stream(stream)))


def cross_attention(q, k, v, kv_len=None, scale=None, y=None, lse=None, workspace=None, stream=None):
    """Attention to an encoder's states: q [B,T,Hq,d], k/v [B,S,Hkv,d] -> y [B,T,Hq,d] in q's dtype.

    Every query of sequence b reads the keys s < kv_len[b] (int32 [B] on the device; all S if
    None).  scale is 1/sqrt(d) if None; a number or a 0-d tensor, read when the call is made.  Any
    strides with contiguous heads, a batch stride of 0 among them (one encoder output for all
    sequences, read as a shared prefix is if kv_len is None).  lse (float32 [B,T,Hq]), if given,
    receives each row's log-sum-exp.  workspace: scratch to use instead of an allocation
    (attention_workspace bytes); calls that may overlap need one each.  Forward only: y carries no
    gradient, whatever the inputs require."""
    return _attention(q, None, None, k, v, kv_len, "kv_len", scale, y, lse, workspace, stream)


def prefix_attention(q, k_prefix, v_prefix, k, v, own_len=None, scale=None, y=None, lse=None, workspace=None,
                     stream=None):
    """Attention of a batch that shares a prefix, whose keys all its sequences read together.

    q [B,T,Hq,d]: the last T tokens of each sequence; k_prefix/v_prefix [P,Hkv,d]; k/v
    [B,L,Hkv,d]: each sequence's own keys, own_len[b] of them (int32 [B]; all L if None).  Query
    t reads the prefix and its own keys s <= own_len[b] - T + t.  The rest as cross_attention."""
    if k_prefix is None or v_prefix is None:
        raise TypeError("k_prefix and v_prefix must be torch.Tensors")
    return _attention(q, k_prefix, v_prefix, k, v, own_len, "own_len", scale, y, lse,
                      workspace, stream)


class LolaLayer:
    """One LoLA attention layer state bound to a caller-owned device buffer.

    W: [Hkv, d, Dh] device tensor in the layer dtype (feature-map weights).
    """

    def __init__(self, cfg: LolaConfig, W: torch.Tensor, device="cuda", stream=None):
        self.cfg = cfg
        self.device = torch.device(device)
        self.dtype = _TORCH_DTYPE[cfg.dtype]
        self.D = 2 * cfg.Dh
        self.B = cfg.B                      # sequences that calls process (set_batch, fork)
        self._check_tensor(W, (cfg.Hkv, cfg.d, cfg.Dh), self.dtype, "W")
        self.nbytes = state_bytes(cfg)
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=self.device)
        self._off = (-self.buf.data_ptr()) % 256
        self.handle = c_void_p()
        _check(lib().lola_state_init(byref(cfg), c_void_p(W.data_ptr()),
                                     c_void_p(self.buf.data_ptr() + self._off), self.nbytes,
                                     _stream(stream), byref(self.handle)))

    @property
    def S(self) -> int:
        """Streams (sequences x kv heads) that calls process."""
        return self.B * self.cfg.Hkv

    # -- argument checks (marshalling only) --------------------------------
    def _check_tensor(self, x, shape, dtype, name, device=None):
        dev = self.device if device is None else device
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if tuple(x.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
        if x.dtype != dtype:
            raise ValueError(f"{name}: dtype {x.dtype}, expected {dtype}")
        if x.device.type != dev.type or (dev.type == "cuda" and dev.index is not None
                                           and x.device.index != dev.index):
            raise ValueError(f"{name}: on {x.device}, expected {dev}")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _shapes(self, T):
        c, B = self.cfg, self.B
        if T is None:
            return (B, c.Hq, c.d), (B, c.Hkv, c.d)
        return (B, T, c.Hq, c.d), (B, T, c.Hkv, c.d)

    # -- calls --------------------------------------------------------------
    def prefill(self, q, k, v, y=None, stream=None) -> torch.Tensor:
        """Chunkwise prefill of T tokens: q [B,T,Hq,d], k/v [B,T,Hkv,d] -> y [B,T,Hq,d] f32."""
        T = q.shape[1]
        sq, sk = self._shapes(T)
        self._check_tensor(q, sq, self.dtype, "q")
        self._check_tensor(k, sk, self.dtype, "k")
        self._check_tensor(v, sk, self.dtype, "v")
        if y is None:
            y = torch.empty(sq, dtype=torch.float32, device=self.device)
        self._check_tensor(y, sq, torch.float32, "y")
        _check(lib().lola_prefill_chunked(self.handle, c_void_p(q.data_ptr()), c_void_p(k.data_ptr()),
                                          c_void_p(v.data_ptr()), T, c_void_p(y.data_ptr()),
                                          _stream(stream)))
        return y

    def decode(self, q, k, v, y=None, stream=None) -> torch.Tensor:
        """One decode step: q [B,Hq,d], k/v [B,Hkv,d] -> y [B,Hq,d] f32."""
        sq, sk = self._shapes(None)
        self._check_tensor(q, sq, self.dtype, "q")
        self._check_tensor(k, sk, self.dtype, "k")
        self._check_tensor(v, sk, self.dtype, "v")
        if y is None:
            y = torch.empty(sq, dtype=torch.float32, device=self.device)
        self._check_tensor(y, sq, torch.float32, "y")
        _check(lib().lola_decode_step(self.handle, c_void_p(q.data_ptr()), c_void_p(k.data_ptr()),
                                      c_void_p(v.data_ptr()), c_void_p(y.data_ptr()), _stream(stream)))
        return y

    def prefill_host(self, q, k, v, y, stream=None) -> torch.Tensor:
        """prefill() with pinned host tensors; copies run inside the library call."""
        cpu = torch.device("cpu")
        T = q.shape[1]
        sq, sk = self._shapes(T)
        for x, s, dt, n in ((q, sq, self.dtype, "q"), (k, sk, self.dtype, "k"), (v, sk, self.dtype, "v"),
                            (y, sq, torch.float32, "y")):
            self._check_tensor(x, s, dt, n, device=cpu)
            if not x.is_pinned():
                raise ValueError(f"{n} must be pinned host memory")
        _check(lib().lola_prefill_chunked_host(self.handle, c_void_p(q.data_ptr()), c_void_p(k.data_ptr()),
                                               c_void_p(v.data_ptr()), T, c_void_p(y.data_ptr()),
                                               _stream(stream)))
        return y

    def decode_host(self, q, k, v, y, stream=None) -> torch.Tensor:
        cpu = torch.device("cpu")
        sq, sk = self._shapes(None)
        for x, s, dt, n in ((q, sq, self.dtype, "q"), (k, sk, self.dtype, "k"), (v, sk, self.dtype, "v"),
                            (y, sq, torch.float32, "y")):
            self._check_tensor(x, s, dt, n, device=cpu)
            if not x.is_pinned():
                raise ValueError(f"{n} must be pinned host memory")
        _check(lib().lola_decode_step_host(self.handle, c_void_p(q.data_ptr()), c_void_p(k.data_ptr()),
                                           c_void_p(v.data_ptr()), c_void_p(y.data_ptr()), _stream(stream)))
        return y

    def set_read_options(self, read_mask: int = 0, decode_update_first: bool = False) -> None:
        """Hide memory branches from later reads (READ_HIDE_* bits); update-first decode order."""
        _check(lib().lola_set_read_options(self.handle, int(read_mask), 1 if decode_update_first else 0))

    def set_batch(self, n: int) -> None:
        """Process only the first n sequences; only before the first token."""
        _check(lib().lola_set_batch(self.handle, int(n)))
        self.B = int(n)

    def fork(self, parents: torch.Tensor, src: "LolaLayer | None" = None, stream=None) -> None:
        """Sequence b becomes a copy of sequence parents[b] of `src` (of this layer itself if None).

        parents: int32 [n] on the layer's device; the layer then holds n sequences.  A parent
        outside src's sequences is reported by check()."""
        src = self if src is None else src
        if not isinstance(src, LolaLayer):
            raise TypeError("src must be a LolaLayer")
        if not isinstance(parents, torch.Tensor) or parents.dim() != 1:
            raise TypeError("parents must be a 1-d torch.Tensor")
        n = parents.shape[0]
        self._check_tensor(parents, (n,), torch.int32, "parents", device=self.buf.device)
        if src.buf.device != self.buf.device:
            raise ValueError(f"src is on {src.buf.device}, expected {self.buf.device}")
        if torch.cuda.current_device() != self.buf.device.index:
            with torch.cuda.device(self.buf.device):
                return self.fork(parents, src, stream)
        _check(lib().lola_state_fork(self.handle, src.handle, c_void_p(parents.data_ptr()), n, _stream(stream)))
        self.B = n

    def set_scorer(self, scorer) -> None:
        """Scoring rule (a name from SCORERS or its LOLA_SCORE_* number); only before the first token."""
        code = SCORERS.index(scorer) if isinstance(scorer, str) else int(scorer)
        _check(lib().lola_set_scorer(self.handle, code))

    def sre_map(self, k, v, sre=None, rel=None, stream=None):
        """SRE of every folded pair at each state time of the last prefill call, and its change
        since first write: k/v [B,T,Hkv,d] (every position so far) -> sre, rel [B,Hkv,n+1,T] f32."""
        c = self.cfg
        T = k.shape[1]
        _, sk = self._shapes(T)
        self._check_tensor(k, sk, self.dtype, "k")
        self._check_tensor(v, sk, self.dtype, "v")
        v_ = LolaStateView()
        _check(lib().lola_state_export(self.handle, byref(v_)))
        shape = (self.B, c.Hkv, max(v_.trace_len, 1), T)
        if sre is None:
            sre = torch.empty(shape, dtype=torch.float32, device=self.device)
        if rel is None:
            rel = torch.empty(shape, dtype=torch.float32, device=self.device)
        self._check_tensor(sre, shape, torch.float32, "sre")
        self._check_tensor(rel, shape, torch.float32, "rel")
        _check(lib().lola_sre_map(self.handle, c_void_p(k.data_ptr()), c_void_p(v.data_ptr()), T,
                                  c_void_p(sre.data_ptr()), c_void_p(rel.data_ptr()), _stream(stream)))
        return sre, rel

    def profile(self, on: bool = True) -> None:
        """Bracket every kernel launch of this layer with CUDA events (tracing aid)."""
        _check(lib().lola_profile_enable(self.handle, 1 if on else 0))

    def profile_read(self) -> dict:
        """{class: (ms, launches)} accumulated since the last read (waits for the events)."""
        n = len(KERNEL_CLASSES)
        ms = (ctypes.c_float * n)()
        cnt = (c_longlong * n)()
        _check(lib().lola_profile_read(self.handle, ms, cnt, n))
        return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_CLASSES)}

    def check(self, stream=None) -> None:
        """Sync point: wait for the stream and raise LolaError if a bounded device-side wait of this
        state gave up (LOLA_ERR_TIMEOUT) or a fork into it had a parent outside its source
        (LOLA_ERR_INVALID_ARG) since the last reset."""
        _check(lib().lola_state_check(self.handle, _stream(stream)))

    def reset(self, stream=None) -> None:
        _check(lib().lola_state_reset(self.handle, _stream(stream)))
        self.B = self.cfg.B

    # -- state views ----------------------------------------------------------
    def _view(self, ptr, shape, dtype):
        n = 1
        for x in shape:
            n *= x
        esize = torch.empty(0, dtype=dtype).element_size()
        off = ptr - self.buf.data_ptr()
        assert 0 <= off and off + n * esize <= self.buf.numel()
        return self.buf[off:off + n * esize].view(dtype).view(*shape)

    def export(self) -> dict:
        """Device views (no copy) of the memories and of the last prefill's cache trace."""
        v = LolaStateView()
        _check(lib().lola_state_export(self.handle, byref(v)))
        c, S, D = self.cfg, self.S, self.D
        out = dict(t=v.t, n_cache=v.n_cache, trace_len=v.trace_len, trace_t0=v.trace_t0,
                   H=self._view(v.H, (S, D, c.d), torch.float32),
                   s=self._view(v.s, (S, D), torch.float32),
                   cache_k=self._view(v.cache_k, (S, c.lambda_, c.d), self.dtype),
                   cache_v=self._view(v.cache_v, (S, c.lambda_, c.d), self.dtype),
                   cache_phik=self._view(v.cache_phik, (S, c.lambda_, D), torch.float32),
                   cache_pos=self._view(v.cache_pos, (S, c.lambda_), torch.int32),
                   win_k=self._view(v.win_k, (S, c.eta, c.d), self.dtype),
                   win_v=self._view(v.win_v, (S, c.eta, c.d), self.dtype),
                   win_phik=self._view(v.win_phik, (S, c.eta, D), torch.float32),
                   err_word=self._view(v.err_word, (1,), torch.int32))
        if v.trace_len > 0 and c.lambda_ > 0:
            stride = v.trace_stride
            full = self._view(v.trace_pos, (S, stride), torch.int32)
            out["trace_pos"] = full[:, :v.trace_len * c.lambda_].reshape(S, v.trace_len, c.lambda_)
        return out

    def close(self) -> None:
        if self.handle:
            lib().lola_state_free(self.handle)
            self.handle = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
