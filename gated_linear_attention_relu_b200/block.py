"""Operators of the block around the token mixer, and of its training step: cross attention to an
encoder's states, layer norm, and the global gradient norm with clipping (the ``la_cross_*``,
``la_layernorm_*`` and ``la_*grad_norm`` entry points of include/la.h).

As in ``binding.py``, every step runs in the CUDA library; this module checks shapes, types and
devices (``ValueError``), reads strides and passes pointers.  The library's own checks raise
``LaError``.  Work goes to ``stream``, by default the current stream of the tensors' device; what a
call allocates (outputs that are not given, a workspace that is not given) belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from dataclasses import dataclass
from typing import Optional

from .binding import LA_BF16, LA_F32, LA_FLAG_FORCE_SIMT, LaError, load

LA_CROSS_FORWARD, LA_CROSS_BACKWARD, LA_CROSS_LENGTHS, LA_CROSS_MASK = 1, 2, 4, 8

_SIZE, _INT, _VP = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p


class LaStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class LaCrossProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "H", "Hkv", "Nq", "Nk")] + [
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
    ] + [(n, LaStrides) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")]


class LaNormProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "groups", "sx", "sy", "sdy", "sdx")] + [
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class LaGrad(ctypes.Structure):
    _fields_ = [("in_", _VP), ("out", _VP), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_declared = False


def _lib():
    global _declared
    lib = load()
    if not _declared:
        C = N = G = _VP  # structs, by reference or as packed bytes
        i64, f32 = ctypes.c_int64, ctypes.c_float
        for name, res, args in (
            ("la_cross_workspace_bytes", _SIZE, [C]),
            ("la_cross_workspace_bytes_for", _SIZE, [C, _INT]),
            ("la_cross_workspace_bytes_of", _SIZE, [C, ctypes.c_uint, _INT]),
            ("la_cross_forward", _INT, [C] + [_VP] * 8 + [_SIZE, _VP]),
            ("la_cross_backward", _INT, [C] + [_VP] * 12 + [_SIZE, _VP]),
            ("la_layernorm_workspace_bytes", _SIZE, [N]),
            ("la_layernorm_workspace_bytes_for", _SIZE, [N, _INT]),
            ("la_layernorm_forward", _INT, [N] + [_VP] * 7),
            ("la_layernorm_backward", _INT, [N] + [_VP] * 9 + [_SIZE, _VP]),
            ("la_clip_workspace_bytes", _SIZE, [i64]),
            ("la_clip_workspace_bytes_for", _SIZE, [i64, _INT]),
            ("la_grad_norm", _INT, [G, i64, _VP, _VP, _SIZE, _VP]),
            ("la_clip_grad_norm", _INT, [G, i64, f32, _VP, _VP, _SIZE, _VP]),
        ):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _declared = True
    return lib


@functools.cache
def _calls():
    """The CPython module that checks tensors and makes the calls (csrc/marshal.cpp), bound to the
    library that is loaded; built if it is missing."""
    import torch  # noqa: F401  (the module links against it)

    from . import build

    module, lib = build.load_marshal(), _lib()
    module.bind(*(ctypes.cast(getattr(lib, name), _VP).value for name in (
        "la_cross_workspace_bytes_of", "la_cross_forward", "la_cross_backward", "la_layernorm_workspace_bytes",
        "la_layernorm_forward", "la_layernorm_backward", "la_clip_workspace_bytes", "la_grad_norm",
        "la_clip_grad_norm")))
    return module


def _on(stream, device, call, *args):
    """``call(*args)`` with ``stream`` current (which is where the module's calls and allocations go)."""
    import torch

    if stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return call(*args)


def _result(r, where):
    """What a call returned; a status in its place is an error."""
    if type(r) is int:
        raise LaError(r, where)
    return r


# ------------------------------------------------------------------------------- cross attention
@dataclass(frozen=True)
class CrossProblem:
    """Sizes and parameters of a cross-attention call (mirrors ``la_cross_problem``; strides are
    read from the tensors).  ``Hkv`` defaults to ``H``, ``scale`` to 1/sqrt(d)."""

    B: int
    H: int
    Nq: int
    Nk: int
    d: int = 128
    Hkv: Optional[int] = None
    scale: Optional[float] = None
    dtype: str = "bf16"
    force_simt: bool = False

    @property
    def kv_heads(self) -> int:
        return self.H if self.Hkv is None else self.Hkv

    @functools.cached_property
    def _head(self) -> bytes:
        """The struct up to the strides."""
        scale = self.d ** -0.5 if self.scale is None else self.scale
        return struct.pack("=5q2ifI", self.B, self.H, self.kv_heads, self.Nq, self.Nk, self.d,
                           LA_BF16 if self.dtype == "bf16" else LA_F32, float(scale),
                           LA_FLAG_FORCE_SIMT if self.force_simt else 0)

    def c(self, **strides) -> LaCrossProblem:
        """The C struct; a tensor (q, k, v, o, dout, dq, dk, dv) whose strides are not given is dense."""
        c = LaCrossProblem.from_buffer_copy(self._head + bytes(ctypes.sizeof(LaCrossProblem) - len(self._head)))
        for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
            keys = name in ("k", "v", "dk", "dv")
            heads, n = (self.kv_heads, self.Nk) if keys else (self.H, self.Nq)
            setattr(c, name, LaStrides(*strides.get(name, (heads * n * self.d, n * self.d, self.d))))
        return c


def cross_workspace_bytes(p: CrossProblem, sm_count: Optional[int] = None, backward: bool = True,
                          padded: bool = True) -> int:
    """Bytes for ``cross_forward`` and, with ``backward``, ``cross_backward``; with ``padded`` they may be
    given a ``kv_len`` or ``key_mask``."""
    uses = LA_CROSS_FORWARD | (LA_CROSS_BACKWARD if backward else 0) | (LA_CROSS_LENGTHS | LA_CROSS_MASK if padded else 0)
    if sm_count is not None and sm_count <= 0:
        return 0
    return int(_lib().la_cross_workspace_bytes_of(ctypes.byref(p.c()), uses, int(sm_count or 0)))


def cross_workspace(p: CrossProblem, device="cuda", backward: bool = True, padded: bool = True):
    """A workspace for ``cross_forward`` and ``cross_backward`` (a program that only serves needs far less
    with ``backward`` False).  Calls that may run at the same time (other streams, captured graphs) need
    workspaces of their own."""
    import torch

    with torch.cuda.device(torch.device(device)):
        n = cross_workspace_bytes(p, backward=backward, padded=padded)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def cross_forward(p: CrossProblem, Q, K, V, kv_len=None, key_mask=None, O=None, lse=None, return_lse=False,
                  ws=None, stream=None):
    """Cross attention of Q [B,H,Nq,d] to K, V [B,Hkv,Nk,d] (strided views are fine: rows of d
    contiguous channels, strides of a multiple of 16 bytes).  ``kv_len`` [B] int32: the first
    kv_len[b] keys are attended; ``key_mask`` [B,Nk] bool: the keys that are.  Returns O, or
    (O, lse [B,H,Nq] fp32) with ``return_lse``; a new O has Q's order of dimensions."""
    args = (p._head, Q, K, V, kv_len, key_mask, O, lse, return_lse, ws)
    call = _calls().cross_forward
    return _result(call(*args) if stream is None else _on(stream, Q.device, call, *args), "la_cross_forward")


def cross_backward(p: CrossProblem, Q, K, V, O, lse, dO, kv_len=None, key_mask=None, grads=None, ws=None, stream=None):
    """Gradients (dQ, dK, dV) of ``cross_forward`` given its O and lse and the output gradient dO."""
    args = (p._head, Q, K, V, O, lse, dO, kv_len, key_mask, *(grads or (None, None, None)), ws)
    call = _calls().cross_backward
    return _result(call(*args) if stream is None else _on(stream, Q.device, call, *args), "la_cross_backward")



# ------------------------------------------------------------------------------- layer norm
@dataclass(frozen=True)
class NormProblem:
    """Sizes and parameters of a layer-norm call (mirrors ``la_norm_problem``).  ``groups``: rows
    are split into that many consecutive groups, each with its own weight and bias."""

    rows: int
    cols: int
    groups: int = 1
    eps: float = 1e-6
    dtype: str = "bf16"

    @functools.cached_property
    def _packed(self) -> bytes:
        """The struct's bytes, for dense tensors."""
        return struct.pack("=7qfiI4x", self.rows, self.cols, self.groups, *(4 * (self.cols,)), self.eps,
                           LA_BF16 if self.dtype == "bf16" else LA_F32, 0)

    def c(self) -> LaNormProblem:
        """The C struct for dense tensors."""
        return LaNormProblem.from_buffer_copy(self._packed)


def layernorm_workspace_bytes(p: NormProblem, sm_count: Optional[int] = None) -> int:
    lib, c = _lib(), p.c()
    if sm_count is None:
        return int(lib.la_layernorm_workspace_bytes(ctypes.byref(c)))
    return int(lib.la_layernorm_workspace_bytes_for(ctypes.byref(c), int(sm_count)))


def layernorm_workspace(p: NormProblem, device="cuda"):
    """A workspace for ``layernorm_backward``."""
    import torch

    with torch.cuda.device(torch.device(device)):
        return torch.empty(max(layernorm_workspace_bytes(p), 16), dtype=torch.uint8, device=device)


def layernorm_forward(p: NormProblem, x, weight=None, bias=None, y=None, mean=None, rstd=None, return_stats=False,
                      stream=None):
    """y = (x - mean) rstd weight_g + bias_g over the rows of x [rows, cols] (row strides are fine).
    ``weight``, ``bias``: fp32 [groups, cols] ([cols] with one group) or None.  ``y`` may be ``x``.
    Returns y, or (y, mean, rstd) ([rows] fp32) with ``return_stats``."""
    args = (p._packed, x, weight, bias, y, mean, rstd, return_stats)
    call = _calls().layernorm_forward
    return _result(call(*args) if stream is None else _on(stream, x.device, call, *args), "la_layernorm_forward")


def layernorm_backward(p: NormProblem, x, dy, mean, rstd, weight=None, dx=None, dweight=None, dbias=None,
                       param_grads=True, ws=None, stream=None):
    """(dx, dweight, dbias) of ``layernorm_forward``; dweight and dbias are fp32 [groups, cols], or
    None with ``param_grads`` False (then only those given are computed).  ``dx`` may be ``dy``."""
    args = (p._packed, x, dy, mean, rstd, weight, dx, dweight, dbias, param_grads, ws)
    call = _calls().layernorm_backward
    return _result(call(*args) if stream is None else _on(stream, x.device, call, *args), "la_layernorm_backward")



# ------------------------------------------------------------------------------- gradient clipping
def _norm_call(tensors, max_norm, out, norm, ws, stream, where):
    tensors = list(tensors)
    args = (tensors, None if out is None else list(out), max_norm, norm, ws)
    call = _calls().clip
    if stream is None:
        return _result(call(*args), where)
    return _result(_on(stream, tensors[0].device if tensors else stream.device, call, *args), where)


def grad_norm(tensors, norm=None, ws=None, stream=None):
    """The 2-norm over all elements of a list of contiguous bf16 / fp32 tensors, as a fp32 scalar
    tensor (``norm`` if given)."""
    return _norm_call(tensors, None, None, norm, ws, stream, "la_grad_norm")


def clip_grad_norm(tensors, max_norm, out=None, norm=None, ws=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of
    ``out``, and returns their norm before that.  Nothing is copied to the host."""
    if max_norm is None:
        raise ValueError("max_norm: a number is expected")
    return _norm_call(tensors, max_norm, out, norm, ws, stream, "la_clip_grad_norm")
