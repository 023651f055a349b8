"""Thin ctypes binding of ``libosdn.so`` (include/osdn.h).

Argument marshalling only: every step of the forward pass and of its
gradients runs in the CUDA kernels behind the C ABI.  PyTorch provides device memory and the stream.
There is no CPU path: if the library is not built, or the tensors are not
on a CUDA device, the calls raise.

The C ABI takes plain pointers, so it cannot see shapes, dtypes or devices;
the binding checks them (every tensor's shape, dtype and device against the
call's layout) before any pointer leaves Python, and runs the call with the
tensors' device current and, by default, on its current stream.  A tensor
of the wrong type would otherwise be read or written out of its bounds.

Every call takes ``stream`` (None: torch's current stream).  A call with a
stream is the call under ``torch.cuda.stream(stream)``: its kernels run there
and what it allocates belongs to that stream.  As with any tensor, the caller
orders the inputs, and a workspace used on several streams, with it.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import inspect
import operator
import os
import threading

import torch

from . import build as _build

OSDN_F32, OSDN_BF16 = 0, 1
ACTS = {"none": 0, "silu": 1, "sigmoid": 2}
STATUS_BYTES = 256
_lock = threading.Lock()
_lib = None

_SIGS = {
    "osdn_version": (ctypes.c_int, []),
    "osdn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "osdn_precond_scan_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "osdn_chunk_fwd_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "osdn_workspace_init": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_check_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "osdn_precond_scan": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 3 +
                          [ctypes.c_float] + [ctypes.c_void_p] * 4 +
                          [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_precond_scan_residual": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 3 +
                                   [ctypes.c_float] + [ctypes.c_void_p] * 5 +
                                   [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_chunk_fwd": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 10 +
                       [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_precond_scan_noalloc": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 3 +
                                  [ctypes.c_float] + [ctypes.c_void_p] * 4),
    "osdn_decode_step": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 5 +
                         [ctypes.c_float] + [ctypes.c_void_p] * 6 +
                         [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_backward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 5),
    "osdn_backward": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 6 +
                      [ctypes.c_float] + [ctypes.c_void_p] * 17 +
                      [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_backward_kda_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 5),
    "osdn_backward_kda": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 6 +
                          [ctypes.c_float] + [ctypes.c_void_p] * 17 +
                          [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_decode_step_kda": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 5 +
                             [ctypes.c_float] + [ctypes.c_void_p] * 6 +
                             [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_chunk_fwd_kda_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "osdn_forward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "osdn_forward": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 5 + [ctypes.c_float] +
                     [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_chunk_fwd_kda": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 10 +
                           [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_decay_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "osdn_decay_attn": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 8 +
                        [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_decay_attn_step": (ctypes.c_int, [ctypes.c_int] * 5 + [ctypes.c_void_p] * 7 +
                             [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_decay_attn_backward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "osdn_decay_attn_backward": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 12 +
                                 [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_group_norm": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 4 +
                        [ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]),
    "osdn_group_norm_backward_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "osdn_group_norm_backward": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.c_void_p] * 5 +
                                 [ctypes.c_int, ctypes.c_float] + [ctypes.c_void_p] * 5 +
                                 [ctypes.c_size_t, ctypes.c_void_p]),
    "osdn_clip_grad_norm_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "osdn_clip_grad_norm": (ctypes.c_int, [ctypes.c_int] + [ctypes.c_void_p] * 4 +
                            [ctypes.c_float] + [ctypes.c_void_p] * 2 +
                            [ctypes.c_size_t, ctypes.c_void_p]),
}


class OsdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (%d)" % (where, status_string(code), code))


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError("libosdn.so is not built (%s): run "
                                   "`python -m preconditioned_delta_rule_phase1_gb300.build`" % path)
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype, fn.argtypes = res, args
            _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().osdn_status_string(int(code)).decode()


def _io(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return OSDN_F32
    if t.dtype == torch.bfloat16:
        return OSDN_BF16
    raise TypeError("io tensors must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("OSDN operates on CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("OSDN needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    _same_device(stream, device)
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _same_device(stream, device):
    if stream is not None and device is not None and stream.device != device:
        raise ValueError("stream is on %s; the call runs on %s" % (stream.device, device))


def _current(stream):
    """The context in which `stream` (None: no change) is torch's current stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _on_stream(fn):
    """`fn` with ``stream=s`` as if called under ``torch.cuda.stream(s)``: what it allocates (its
    outputs, a workspace of its own or a grown one) belongs to that stream too, so that nothing is
    filled, or handed on to another tensor, on a stream that the kernels are not ordered with."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        with _current(stream):
            return fn(*args, **kw)
    return call


F32 = torch.float32


def _expect(name, t, shape, dtype, device):
    """Raise unless `t` (a tensor, or None for an absent optional argument)
    has the shape, dtype and device the call reads or writes, and is dense."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != device:
        raise ValueError("%s is on %s; the call runs on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (the library reads it densely)" % name)


def _on(device):
    """The context of a call on `device`: that CUDA device current."""
    if device.type != "cuda":
        raise ValueError("OSDN operates on CUDA tensors only")
    return torch.cuda.device(device)


def _workspace(workspace, device):
    ws = workspace or Workspace(device=device)
    if ws.buf.device != device:
        raise ValueError("workspace is on %s; the call runs on %s" % (ws.buf.device, device))
    return ws


def _check(code: int, where: str):
    if code != 0:
        raise OsdnError(code, where)


class Workspace:
    """A caller-owned device workspace (status word + per-call scratch)."""

    def __init__(self, nbytes: int = STATUS_BYTES, device=None, stream=None):
        self.device = torch.device(device or "cuda")
        self.buf = torch.empty(0, dtype=torch.uint8, device=self.device)
        self.ensure(max(nbytes, STATUS_BYTES), stream)

    def ensure(self, nbytes: int, stream=None):
        """At least `nbytes` bytes, allocated and zeroed on `stream` (None: the current one)."""
        if self.buf.numel() < nbytes:
            old = self.buf
            with _current(stream):
                self.buf = torch.zeros(((nbytes + 255) // 256) * 256, dtype=torch.uint8,
                                       device=self.device)
                if old.numel() >= STATUS_BYTES:  # keep a sticky status already raised
                    self.buf[:STATUS_BYTES].copy_(old[:STATUS_BYTES])
                    if old.is_cuda:  # it may belong to another stream, and is in use on this one
                        old.record_stream(torch.cuda.current_stream(old.device))
        return self

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def reset(self, stream=None):
        _check(lib().osdn_workspace_init(self.ptr, self.nbytes, _stream(stream)), "workspace_init")

    def status(self, stream=None) -> int:
        return lib().osdn_check_status(self.ptr, _stream(stream))


def precond_scan_workspace_bytes(B, H, T, K) -> int:
    return int(lib().osdn_precond_scan_workspace_bytes(B, H, T, K))


def chunk_fwd_workspace_bytes(io, B, H, T, K, V) -> int:
    return int(lib().osdn_chunk_fwd_workspace_bytes(io, B, H, T, K, V))


def forward_workspace_bytes(io, B, H, T, K, V) -> int:
    return int(lib().osdn_forward_workspace_bytes(io, B, H, T, K, V))


def backward_workspace_bytes(B, H, T, K, V) -> int:
    return int(lib().osdn_backward_workspace_bytes(B, H, T, K, V))


def backward_kda_workspace_bytes(B, H, T, K, V) -> int:
    return int(lib().osdn_backward_kda_workspace_bytes(B, H, T, K, V))


@_on_stream
def precond_scan(k, beta, r=None, eta=0.1, d0=None, ktilde=None, dT=None, workspace=None,
                 stream=None, log_ratio=None):
    """Phase 1 (osdn_precond_scan): returns (ktilde, dT).

    With ``log_ratio`` (True, or a [B, H] fp32 tensor to fill) the call goes
    through osdn_precond_scan_residual and returns (ktilde, dT, log_ratio):
    per sequence sum_t log((1 - beta_t <d_t, k_t^2>)^2).
    """
    B, H, T, K = k.shape
    io, dev = _io(k), k.device
    _expect("beta", beta, (B, H, T), F32, dev)
    _expect("r", r, (B, H, T), F32, dev)
    _expect("d0", d0, (B, H, K), F32, dev)
    if ktilde is None:
        ktilde = torch.empty_like(k)
    if dT is None:
        dT = torch.empty(B, H, K, dtype=F32, device=dev)
    _expect("ktilde", ktilde, (B, H, T, K), k.dtype, dev)
    _expect("dT", dT, (B, H, K), F32, dev)
    residual = not (log_ratio is None or log_ratio is False)
    if log_ratio is True:
        log_ratio = torch.empty(B, H, dtype=F32, device=dev)
    if residual:
        _expect("log_ratio", log_ratio, (B, H), F32, dev)
    ws = _workspace(workspace, dev)
    with _on(dev):
        ws.ensure(precond_scan_workspace_bytes(B, H, T, K))
        if not residual:
            code = lib().osdn_precond_scan(io, B, H, T, K, _ptr(k), _ptr(beta), _ptr(r),
                                           float(eta), _ptr(d0), _ptr(ktilde), _ptr(dT), ws.ptr,
                                           ws.nbytes, _stream(stream, dev))
            _check(code, "osdn_precond_scan")
            return ktilde, dT
        code = lib().osdn_precond_scan_residual(io, B, H, T, K, _ptr(k), _ptr(beta), _ptr(r),
                                                float(eta), _ptr(d0), _ptr(ktilde), _ptr(dT),
                                                _ptr(log_ratio), ws.ptr, ws.nbytes,
                                                _stream(stream, dev))
    _check(code, "osdn_precond_scan_residual")
    return ktilde, dT, log_ratio


@_on_stream
def precond_scan_noalloc(k, beta, r=None, eta=0.1, d0=None, ktilde=None, dT=None, stream=None):
    """Phase 1 through osdn_precond_scan_noalloc: no workspace, no device
    allocation inside the call (outputs are allocated here only when not given)."""
    B, H, T, K = k.shape
    io, dev = _io(k), k.device
    _expect("beta", beta, (B, H, T), F32, dev)
    _expect("r", r, (B, H, T), F32, dev)
    _expect("d0", d0, (B, H, K), F32, dev)
    if ktilde is None:
        ktilde = torch.empty_like(k)
    if dT is None:
        dT = torch.empty(B, H, K, dtype=F32, device=dev)
    _expect("ktilde", ktilde, (B, H, T, K), k.dtype, dev)
    _expect("dT", dT, (B, H, K), F32, dev)
    with _on(dev):
        code = lib().osdn_precond_scan_noalloc(io, B, H, T, K, _ptr(k), _ptr(beta), _ptr(r),
                                               float(eta), _ptr(d0), _ptr(ktilde), _ptr(dT),
                                               _stream(stream, dev))
    _check(code, "osdn_precond_scan_noalloc")
    return ktilde, dT


@_on_stream
def chunk_fwd(q, k, ktilde, v, beta, alpha=None, S0=None, o=None, ST=None, workspace=None,
              stream=None):
    """Phase 2 (osdn_chunk_fwd): returns (o, ST)."""
    B, H, T, K = k.shape
    V = v.shape[-1]
    io, dev = _io(k), k.device
    _expect("q", q, (B, H, T, K), k.dtype, dev)
    _expect("ktilde", ktilde, (B, H, T, K), k.dtype, dev)
    _expect("v", v, (B, H, T, V), k.dtype, dev)
    _expect("beta", beta, (B, H, T), F32, dev)
    _expect("alpha", alpha, (B, H, T), F32, dev)
    _expect("S0", S0, (B, H, V, K), F32, dev)
    if o is None:
        o = torch.empty(B, H, T, V, dtype=k.dtype, device=dev)
    if ST is None:
        ST = torch.empty(B, H, V, K, dtype=F32, device=dev)
    _expect("o", o, (B, H, T, V), k.dtype, dev)
    _expect("ST", ST, (B, H, V, K), F32, dev)
    ws = _workspace(workspace, dev)
    with _on(dev):
        ws.ensure(chunk_fwd_workspace_bytes(io, B, H, T, K, V))
        code = lib().osdn_chunk_fwd(io, B, H, T, K, V, _ptr(q), _ptr(k), _ptr(ktilde), _ptr(v),
                                    _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(ST), ws.ptr,
                                    ws.nbytes, _stream(stream, dev))
    _check(code, "osdn_chunk_fwd")
    return o, ST


@_on_stream
def forward(q, k, v, beta, r=None, eta=0.1, d0=None, alpha=None, S0=None, workspace=None,
            stream=None):
    """Both phases: returns (ktilde, dT, o, ST)."""
    ws = _workspace(workspace, k.device)
    ktilde, dT = precond_scan(k, beta, r, eta, d0, workspace=ws, stream=stream)
    o, ST = chunk_fwd(q, k, ktilde, v, beta, alpha, S0, workspace=ws, stream=stream)
    return ktilde, dT, o, ST


@_on_stream
def forward_fused(q, k, v, beta, r=None, eta=0.1, d0=None, alpha=None, S0=None, o=None, dT=None,
                  ST=None, workspace=None, stream=None):
    """Both phases in one call (osdn_forward), ktilde kept off global memory
    for bf16 I/O: returns (dT, o, ST)."""
    B, H, T, K = k.shape
    V = v.shape[-1]
    io, dev = _io(k), k.device
    _expect("q", q, (B, H, T, K), k.dtype, dev)
    _expect("v", v, (B, H, T, V), k.dtype, dev)
    _expect("beta", beta, (B, H, T), F32, dev)
    _expect("r", r, (B, H, T), F32, dev)
    _expect("d0", d0, (B, H, K), F32, dev)
    _expect("alpha", alpha, (B, H, T), F32, dev)
    _expect("S0", S0, (B, H, V, K), F32, dev)
    if o is None:
        o = torch.empty(B, H, T, V, dtype=k.dtype, device=dev)
    if dT is None:
        dT = torch.empty(B, H, K, dtype=F32, device=dev)
    if ST is None:
        ST = torch.empty(B, H, V, K, dtype=F32, device=dev)
    _expect("o", o, (B, H, T, V), k.dtype, dev)
    _expect("dT", dT, (B, H, K), F32, dev)
    _expect("ST", ST, (B, H, V, K), F32, dev)
    ws = _workspace(workspace, dev)
    with _on(dev):
        ws.ensure(forward_workspace_bytes(io, B, H, T, K, V))
        code = lib().osdn_forward(io, B, H, T, K, V, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r),
                                  float(eta), _ptr(d0), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(dT),
                                  _ptr(ST), ws.ptr, ws.nbytes, _stream(stream, dev))
    _check(code, "osdn_forward")
    return dT, o, ST


@_on_stream
def decode_step(q, k, v, beta, d, S, r=None, eta=0.1, alpha=None, o=None, ktilde=None,
                workspace=None, stream=None):
    """One recurrent step (osdn_decode_step): updates d [B,H,K] and S [B,H,V,K]
    (fp32) in place for the token q, k [B,H,K], v [B,H,V] (io); returns
    (o, ktilde)."""
    return _decode(False, q, k, v, beta, d, S, r, eta, alpha, o, ktilde, workspace, stream)


@_on_stream
def decode_step_kda(q, k, v, beta, d, S, r=None, eta=0.1, alpha_k=None, o=None, ktilde=None,
                    workspace=None, stream=None):
    """One recurrent step with a decay per key channel (osdn_decode_step_kda):
    as ``decode_step``, with alpha_k [B,H,K] fp32."""
    return _decode(True, q, k, v, beta, d, S, r, eta, alpha_k, o, ktilde, workspace, stream)


def _decode(per_channel, q, k, v, beta, d, S, r, eta, alpha, o, ktilde, workspace, stream):
    B, H, K = k.shape
    V = v.shape[-1]
    io, dev = _io(k), k.device
    _expect("q", q, (B, H, K), k.dtype, dev)
    _expect("v", v, (B, H, V), k.dtype, dev)
    _expect("beta", beta, (B, H), F32, dev)
    _expect("r", r, (B, H), F32, dev)
    _expect("alpha", alpha, (B, H, K) if per_channel else (B, H), F32, dev)
    _expect("d", d, (B, H, K), F32, dev)
    _expect("S", S, (B, H, V, K), F32, dev)
    if o is None:
        o = torch.empty(B, H, V, dtype=k.dtype, device=dev)
    if ktilde is None:
        ktilde = torch.empty(B, H, K, dtype=k.dtype, device=dev)
    _expect("o", o, (B, H, V), k.dtype, dev)
    _expect("ktilde", ktilde, (B, H, K), k.dtype, dev)
    ws = _workspace(workspace, dev)
    name = "osdn_decode_step_kda" if per_channel else "osdn_decode_step"
    with _on(dev):
        code = getattr(lib(), name)(io, B, H, K, V, _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                    _ptr(r), float(eta), _ptr(alpha), _ptr(d), _ptr(S), _ptr(o),
                                    _ptr(ktilde), ws.ptr, ws.nbytes, _stream(stream, dev))
    _check(code, name)
    return o, ktilde


@_on_stream
def backward(q, k, ktilde, v, beta, r=None, eta=0.1, d0=None, alpha=None, S0=None, *, do=None,
             dST=None, ddT=None, dktilde=None, workspace=None, stream=None):
    """Gradients of both phases (osdn_backward).

    Takes the forward's inputs, the ktilde it produced and the cotangents of
    its outputs (o, ST, dT, ktilde; None counts as zero).  Returns a dict
    keyed like the inputs: q, k, v, beta (io / fp32), eta ([B, H]: each
    sequence's share; the scalar gradient is the sum), and r, alpha, d0, S0
    for those given (an input given as None has no entry).
    """
    return _backward(False, q, k, ktilde, v, beta, r, eta, d0, alpha, S0, do, dST, ddT, dktilde,
                     workspace, stream)


@_on_stream
def backward_kda(q, k, ktilde, v, beta, r=None, eta=0.1, d0=None, alpha_k=None, S0=None, *,
                 do=None, dST=None, ddT=None, dktilde=None, workspace=None, stream=None):
    """Gradients of both phases with a decay per key channel
    (osdn_backward_kda): as ``backward``, with alpha_k [B, H, T, K] and its
    gradient under the key "alpha" ([B, H, T, K])."""
    return _backward(True, q, k, ktilde, v, beta, r, eta, d0, alpha_k, S0, do, dST, ddT,
                     dktilde, workspace, stream)


def _backward(per_channel, q, k, ktilde, v, beta, r, eta, d0, alpha, S0, do, dST, ddT, dktilde,
              workspace, stream):
    B, H, T, K = k.shape
    V = v.shape[-1]
    io, dev = _io(k), k.device
    ashape = (B, H, T, K) if per_channel else (B, H, T)
    for name, t, shape, dt in (("q", q, (B, H, T, K), k.dtype),
                               ("ktilde", ktilde, (B, H, T, K), k.dtype),
                               ("v", v, (B, H, T, V), k.dtype),
                               ("beta", beta, (B, H, T), F32), ("r", r, (B, H, T), F32),
                               ("d0", d0, (B, H, K), F32), ("alpha", alpha, ashape, F32),
                               ("S0", S0, (B, H, V, K), F32), ("do", do, (B, H, T, V), k.dtype),
                               ("dST", dST, (B, H, V, K), F32), ("ddT", ddT, (B, H, K), F32),
                               ("dktilde", dktilde, (B, H, T, K), k.dtype)):
        _expect(name, t, shape, dt, dev)
    if q is None or ktilde is None or v is None or beta is None:
        raise ValueError("q, ktilde, v and beta are required")
    new = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device=dev)
    g = {"q": new(B, H, T, K, dtype=k.dtype), "k": new(B, H, T, K, dtype=k.dtype),
         "v": new(B, H, T, V, dtype=k.dtype), "beta": new(B, H, T), "eta": new(B, H)}
    if r is not None:
        g["r"] = new(B, H, T)
    if alpha is not None:
        g["alpha"] = new(*ashape)
    if d0 is not None:
        g["d0"] = new(B, H, K)
    if S0 is not None:
        g["S0"] = new(B, H, V, K)
    ws = _workspace(workspace, dev)
    fn, size = ((lib().osdn_backward_kda, backward_kda_workspace_bytes) if per_channel
                else (lib().osdn_backward, backward_workspace_bytes))
    with _on(dev):
        ws.ensure(size(B, H, T, K, V))
        code = fn(io, B, H, T, K, V, _ptr(q), _ptr(k), _ptr(ktilde), _ptr(v), _ptr(beta), _ptr(r),
                  float(eta), _ptr(d0), _ptr(alpha), _ptr(S0), _ptr(do), _ptr(dST), _ptr(ddT),
                  _ptr(dktilde), _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"]), _ptr(g["beta"]),
                  _ptr(g.get("r")), _ptr(g.get("alpha")), _ptr(g.get("d0")), _ptr(g.get("S0")),
                  _ptr(g["eta"]), ws.ptr, ws.nbytes, _stream(stream, dev))
    _check(code, "osdn_backward_kda" if per_channel else "osdn_backward")
    return g


@_on_stream
def chunk_fwd_kda(q, k, ktilde, v, beta, alpha_k=None, S0=None, o=None, ST=None, workspace=None,
                  stream=None):
    """Phase 2 with a decay per key channel (osdn_chunk_fwd_kda), alpha_k
    [B, H, T, K] fp32: returns (o, ST)."""
    B, H, T, K = k.shape
    V = v.shape[-1]
    io, dev = _io(k), k.device
    _expect("q", q, (B, H, T, K), k.dtype, dev)
    _expect("ktilde", ktilde, (B, H, T, K), k.dtype, dev)
    _expect("v", v, (B, H, T, V), k.dtype, dev)
    _expect("beta", beta, (B, H, T), F32, dev)
    _expect("alpha_k", alpha_k, (B, H, T, K), F32, dev)
    _expect("S0", S0, (B, H, V, K), F32, dev)
    if o is None:
        o = torch.empty(B, H, T, V, dtype=k.dtype, device=dev)
    if ST is None:
        ST = torch.empty(B, H, V, K, dtype=F32, device=dev)
    _expect("o", o, (B, H, T, V), k.dtype, dev)
    _expect("ST", ST, (B, H, V, K), F32, dev)
    ws = _workspace(workspace, dev)
    with _on(dev):
        ws.ensure(int(lib().osdn_chunk_fwd_kda_workspace_bytes(io, B, H, T, K, V)))
        code = lib().osdn_chunk_fwd_kda(io, B, H, T, K, V, _ptr(q), _ptr(k), _ptr(ktilde),
                                        _ptr(v), _ptr(beta), _ptr(alpha_k), _ptr(S0), _ptr(o),
                                        _ptr(ST), ws.ptr, ws.nbytes, _stream(stream, dev))
    _check(code, "osdn_chunk_fwd_kda")
    return o, ST


@_on_stream
def forward_kda(q, k, v, beta, r=None, eta=0.1, d0=None, alpha_k=None, S0=None, workspace=None,
                stream=None):
    """Both phases with a decay per key channel in Phase 2: returns
    (ktilde, dT, o, ST)."""
    ws = _workspace(workspace, k.device)
    ktilde, dT = precond_scan(k, beta, r, eta, d0, workspace=ws, stream=stream)
    o, ST = chunk_fwd_kda(q, k, ktilde, v, beta, alpha_k, S0, workspace=ws, stream=stream)
    return ktilde, dT, o, ST


# The decayed layer's calls.  Its steps and norms take a few microseconds on the device, so the
# checks above are made in one pass per tensor, and addresses go to ctypes as plain integers.

_IO = {torch.float32: OSDN_F32, torch.bfloat16: OSDN_BF16}
_dtype_of = operator.attrgetter("dtype")


def _arg(name, t, shape, dtype, device):
    """The address of `t` (None for an absent argument) after the checks of ``_expect``."""
    if t is None:
        return None
    try:
        if (t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _expect(name, t, shape, dtype, device)
    raise ValueError("%s does not fit the call" % name)


def _run(name, device, stream, args, workspace=None, size=None):
    """Call `name` with `args`, then the workspace (if given) and the stream, on `device`.
    `size`: the C call, and its arguments, that says how large the workspace has to be."""
    if device.type != "cuda":
        raise ValueError("OSDN operates on CUDA tensors only")
    _same_device(stream, device)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(name, device, stream, args, workspace, size)
    if workspace is not None:
        if size is not None:
            nbytes = _bytes(device.index, *size)
            if workspace.buf.numel() < nbytes:
                workspace.ensure(nbytes)
        args += (workspace.buf.data_ptr(), workspace.buf.numel())
    s = torch.cuda.current_stream(device) if stream is None else stream
    code = getattr(_lib or lib(), name)(*args, s.cuda_stream)
    if code:
        raise OsdnError(code, name)


@functools.lru_cache(maxsize=1024)
def _bytes(device, name, *shape) -> int:
    """What `name` answers on the device numbered `device`, the current one: it may depend on its
    number of SMs."""
    return int(getattr(lib(), name)(*shape))


def decay_attn_workspace_bytes(io, B, H, T, K, V) -> int:
    return int(lib().osdn_decay_attn_workspace_bytes(io, B, H, T, K, V))


def decay_attn_backward_workspace_bytes(io, B, H, T, K, V) -> int:
    return int(lib().osdn_decay_attn_backward_workspace_bytes(io, B, H, T, K, V))


def group_norm_backward_workspace_bytes(B, G, T, D) -> int:
    return int(lib().osdn_group_norm_backward_workspace_bytes(B, G, T, D))


def clip_grad_norm_workspace_bytes(n) -> int:
    return int(lib().osdn_clip_grad_norm_workspace_bytes(n))


@_on_stream
def decay_attn(q, k, v, decay, S0=None, o=None, ST=None, workspace=None, stream=None):
    """Linear attention with a decay per head (osdn_decay_attn), q, k [B,H,T,K],
    v [B,H,T,V] (io), decay [H] fp32 in [0, 1], S0 [B,H,V,K] fp32 or None:
    returns (o, ST)."""
    B, H, T, K = k.shape
    V = v.shape[-1]
    dt, dev = k.dtype, k.device
    io = _io(k)
    qk, vo, st = (B, H, T, K), (B, H, T, V), (B, H, V, K)
    if o is None:
        o = torch.empty(vo, dtype=dt, device=dev)
    if ST is None:
        ST = torch.empty(st, dtype=F32, device=dev)
    args = (io, B, H, T, K, V, _arg("q", q, qk, dt, dev), _arg("k", k, qk, dt, dev),
            _arg("v", v, vo, dt, dev), _arg("decay", decay, (H,), F32, dev),
            _arg("S0", S0, st, F32, dev), _arg("o", o, vo, dt, dev), _arg("ST", ST, st, F32, dev))
    _run("osdn_decay_attn", dev, stream, args, _workspace(workspace, dev),
         ("osdn_decay_attn_workspace_bytes", io, B, H, T, K, V))
    return o, ST


@_on_stream
def decay_attn_step(q, k, v, decay, S, o=None, workspace=None, stream=None):
    """One token of ``decay_attn`` (osdn_decay_attn_step): updates S [B,H,V,K]
    (fp32) in place for the token q, k [B,H,K], v [B,H,V] (io); returns o."""
    B, H, K = k.shape
    V = v.shape[-1]
    dt, dev = k.dtype, k.device
    io = _io(k)
    if o is None:
        o = torch.empty((B, H, V), dtype=dt, device=dev)
    args = (io, B, H, K, V, _arg("q", q, (B, H, K), dt, dev), _arg("k", k, (B, H, K), dt, dev),
            _arg("v", v, (B, H, V), dt, dev), _arg("decay", decay, (H,), F32, dev),
            _arg("S", S, (B, H, V, K), F32, dev), _arg("o", o, (B, H, V), dt, dev))
    _run("osdn_decay_attn_step", dev, stream, args, _workspace(workspace, dev))
    return o


@_on_stream
def decay_attn_backward(q, k, v, decay, S0=None, *, do, dST=None, workspace=None, stream=None):
    """Gradients through ``decay_attn`` (osdn_decay_attn_backward) given the
    cotangents do [B,H,T,V] (io) of o and dST [B,H,V,K] fp32 of ST (None: zero).
    Returns a dict with q, k, v (io) and, if S0 is given, S0 (fp32).  The decay
    is a constant and has no gradient."""
    B, H, T, K = k.shape
    V = v.shape[-1]
    dt, dev = k.dtype, k.device
    io = _io(k)
    qk, vo, st = (B, H, T, K), (B, H, T, V), (B, H, V, K)
    args = (io, B, H, T, K, V, _arg("q", q, qk, dt, dev), _arg("k", k, qk, dt, dev),
            _arg("v", v, vo, dt, dev), _arg("decay", decay, (H,), F32, dev),
            _arg("S0", S0, st, F32, dev), _arg("do", do, vo, dt, dev), _arg("dST", dST, st, F32, dev))
    g = {"q": torch.empty_like(k), "k": torch.empty_like(k), "v": torch.empty_like(v)}
    if S0 is not None:
        g["S0"] = torch.empty_like(S0)
    args += (g["q"].data_ptr(), g["k"].data_ptr(), g["v"].data_ptr(),
             None if S0 is None else g["S0"].data_ptr())
    _run("osdn_decay_attn_backward", dev, stream, args, _workspace(workspace, dev),
         ("osdn_decay_attn_backward_workspace_bytes", io, B, H, T, K, V))
    return g


def _norm_shape(x, groups):
    """(B, G, T, D, heads_first) of a group norm's input: [B,G,T,D] (four
    dimensions), or [B,T,C] with `groups`."""
    if x.dim() == 4:
        B, G, T, D = x.shape
        if groups is not None and groups != G:
            raise ValueError("x has %d groups, groups is %s" % (G, groups))
        return B, G, T, D, 1
    if x.dim() != 3:
        raise ValueError("x must be [B,G,T,D] or [B,T,C], got shape %s" % (tuple(x.shape),))
    B, T, C = x.shape
    if not groups or groups < 0 or C % groups:
        raise ValueError("groups (%s) must divide the %d channels of x" % (groups, C))
    return B, groups, T, C // groups, 0


def _act(act):
    if act not in ACTS:
        raise ValueError("act must be one of %s, got %r" % (sorted(ACTS), act))
    return ACTS[act]


@_on_stream
def group_norm(x, weight=None, bias=None, gate=None, groups=None, act="none", eps=1e-5, y=None,
               stream=None):
    """Group norm of every token with an activation (osdn_group_norm).

    x is the attention's output [B,H,T,D] (a group is a head) or channels last
    [B,T,C] with `groups`; weight, bias [C] fp32; gate [B,T,C] (io).  Returns
    y [B,T,C] = act(norm(x)), or norm(x) act(gate) with a gate; act is "none",
    "silu" or "sigmoid"."""
    a = _act(act)
    B, G, T, D, first = _norm_shape(x, groups)
    io, dt, dev, C = _io(x), x.dtype, x.device, G * D
    if y is None:
        y = torch.empty((B, T, C), dtype=dt, device=dev)
    args = (io, B, G, T, D, first, _arg("x", x, x.shape, dt, dev), _arg("weight", weight, (C,), F32, dev),
            _arg("bias", bias, (C,), F32, dev), _arg("gate", gate, (B, T, C), dt, dev), a, float(eps),
            _arg("y", y, (B, T, C), dt, dev))
    _run("osdn_group_norm", dev, stream, args)
    return y


@_on_stream
def group_norm_backward(x, dy, weight=None, bias=None, gate=None, groups=None, act="none",
                        eps=1e-5, workspace=None, stream=None):
    """Gradients of ``group_norm`` (osdn_group_norm_backward) given dy [B,T,C]:
    a dict with x (in x's layout) and weight, bias, gate for those given."""
    a = _act(act)
    B, G, T, D, first = _norm_shape(x, groups)
    io, dt, dev, C = _io(x), x.dtype, x.device, G * D
    args = (io, B, G, T, D, first, _arg("x", x, x.shape, dt, dev), _arg("dy", dy, (B, T, C), dt, dev),
            _arg("weight", weight, (C,), F32, dev), _arg("bias", bias, (C,), F32, dev),
            _arg("gate", gate, (B, T, C), dt, dev), a, float(eps))
    g = {"x": torch.empty_like(x)}
    for name, t in (("weight", weight), ("bias", bias), ("gate", gate)):
        if t is not None:
            g[name] = torch.empty_like(t)
    at = lambda name: g[name].data_ptr() if name in g else None  # noqa: E731
    args += (at("x"), at("gate"), at("weight"), at("bias"))
    _run("osdn_group_norm_backward", dev, stream, args, _workspace(workspace, dev),
         ("osdn_group_norm_backward_workspace_bytes", B, G, T, D))
    return g


def _tensor_table(what, tensors, dev):
    """Addresses, element counts and io types of `tensors`, which must be dense and on
    `dev`.  Whole-list maps: a model has hundreds of gradients."""
    at, n = (dev.index if dev.type == "cuda" else -1), len(tensors)
    if (list(map(torch.Tensor.get_device, tensors)).count(at) != n
            or not all(map(torch.Tensor.is_contiguous, tensors))):
        for i, t in enumerate(tensors):
            _expect("%s[%d]" % (what, i), t, t.shape, t.dtype, dev)
    try:
        ios = array.array("i", [_IO[d] for d in map(_dtype_of, tensors)])
    except KeyError as e:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (what, e)) from None
    return (array.array("Q", map(torch.Tensor.data_ptr, tensors)),
            array.array("q", map(torch.Tensor.numel, tensors)), ios)


@_on_stream
def clip_grad_norm(grads, max_norm, outs=None, norm=None, workspace=None, stream=None):
    """Clip tensors by their global 2-norm (osdn_clip_grad_norm): every g becomes
    g min(1, max_norm / norm), in place, or in `outs` (as many elements of the
    same types).  Returns norm [1] fp32 on the device.  max_norm = inf: the
    norm alone."""
    grads = list(grads)
    n = len(grads)
    if n == 0 and norm is None:
        raise ValueError("no gradients and no norm tensor: the device is unknown")
    dev = grads[0].device if n else norm.device
    gp, sizes, ios = _tensor_table("grads", grads, dev)
    op = gp
    if outs is not None:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError("%d gradients, %d outputs" % (n, len(outs)))
        op, osizes, oios = _tensor_table("outs", outs, dev)
        if osizes != sizes or oios != ios:
            raise ValueError("outs must have the gradients' sizes and types")
    writes = outs is not None or max_norm != float("inf")
    if writes and len(set(op)) != n:   # empty tensors may share an address
        written = [p for p, s in zip(op, sizes) if s]
        if len(set(written)) != len(written):
            raise ValueError("a tensor is written twice")
    if norm is None:
        norm = torch.empty(1, dtype=F32, device=dev)
    at = lambda a: a.buffer_info()[0] if n else None  # noqa: E731
    args = (n, at(gp), None if outs is None else at(op), at(sizes), at(ios), float(max_norm),
            _arg("norm", norm, (1,), F32, dev))
    _run("osdn_clip_grad_norm", dev, stream, args, _workspace(workspace, dev),
         ("osdn_clip_grad_norm_workspace_bytes", n))
    return norm


@_on_stream
def grad_norm(grads, norm=None, workspace=None, stream=None):
    """The global 2-norm of the tensors, [1] fp32 on the device."""
    return clip_grad_norm(grads, float("inf"), norm=norm, workspace=workspace, stream=stream)
