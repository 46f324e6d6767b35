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
def _lists():
    """The CPython helper that reads a list of tensors (csrc/lists.cpp), built if it is missing."""
    import torch  # noqa: F401  (the helper links against it)

    from . import build

    build.build_lists()
    from . import _lists as helper

    return helper


def _torch_dtype(name: str):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


def _wrong(t, name, shape, dtype, device, dense):
    """Raises the ValueError that says what is wrong with a tensor."""
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, expected {device} (a CUDA device)")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: must be contiguous" if dense else f"{name}: the elements of a row must be contiguous")


def _want(t, name: str, shape, dtype, device):
    """A contiguous CUDA tensor of this shape, type and device, or ValueError."""
    if not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and t.is_contiguous()):
        _wrong(t, name, shape, dtype, device, True)


def _rows(t, name, shape, dtype, device):
    """The same, but only the last dimension need be contiguous.  Returns the strides."""
    st = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_cuda and
            (st[-1] == 1 or shape[-1] <= 1 or t.numel() == 0)):
        _wrong(t, name, shape, dtype, device, False)
    return st


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class _On:
    """Makes ``device`` and ``stream`` current, so that the library's device queries and the caching
    allocator see them; ``handle`` is the stream's.  (A class: entering it costs less than a
    generator.)"""

    __slots__ = ("handle", "guard")

    def __init__(self, device, stream):
        import torch

        self.guard = None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
            self.guard = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        else:
            if torch.cuda.current_device() != device.index:
                self.guard = torch.cuda.device(device)
            # (torch.cuda.current_stream makes a stream object first, which takes longer than the call)
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            return self.guard.__exit__(*exc)
        return None


def _workspace(ws, device, query, *args):
    """(tensor, size): the given workspace, or a new one of the size that ``query(*args)`` says."""
    import torch

    if ws is None:
        n = query(*args)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=device), n
    if ws.device != device or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous uint8 tensor on {device} is expected")
    return ws, ws.numel()


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

    @functools.cached_property
    def _shapes(self):
        return (self.B, self.H, self.Nq, self.d), (self.B, self.kv_heads, self.Nk, self.d)

    def c(self, q=None, k=None, v=None, o=None, dout=None, dq=None, dk=None, dv=None) -> LaCrossProblem:
        """The C struct, from the tensors' strides; None counts as dense."""
        dq_ = (self.H * self.Nq * self.d, self.Nq * self.d, self.d, 1)
        dk_ = (self.kv_heads * self.Nk * self.d, self.Nk * self.d, self.d, 1)
        return LaCrossProblem.from_buffer_copy(self._packed(q or dq_, k or dk_, v or dk_, o or dq_, dout or dq_, dq or dq_,
                                                            dk or dk_, dv or dk_))

    def _packed(self, q, k, v, o, *grads) -> bytes:
        """The struct's bytes, from the strides of four or eight tensors."""
        if not grads:
            return self._head + _STRIDES4(*q[:3], *k[:3], *v[:3], *o[:3]) + _NO_STRIDES
        g, dq, dk, dv = grads
        return (self._head + _STRIDES4(*q[:3], *k[:3], *v[:3], *o[:3]) +
                _STRIDES4(*g[:3], *dq[:3], *dk[:3], *dv[:3]))


_STRIDES4 = struct.Struct("=12q").pack
_NO_STRIDES = bytes(96)


def cross_workspace_bytes(p: CrossProblem, sm_count: Optional[int] = None) -> int:
    lib, c = _lib(), p.c()
    if sm_count is None:
        return int(lib.la_cross_workspace_bytes(ctypes.byref(c)))
    return int(lib.la_cross_workspace_bytes_for(ctypes.byref(c), int(sm_count)))


def cross_workspace(p: CrossProblem, device="cuda"):
    """A workspace for ``cross_forward`` and ``cross_backward``.  Calls that may run at the same
    time (other streams, captured graphs) need workspaces of their own."""
    import torch

    with torch.cuda.device(torch.device(device)):
        n = cross_workspace_bytes(p)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _cross_masks(p: CrossProblem, kv_len, key_mask, device):
    import torch

    if kv_len is not None:
        _want(kv_len, "kv_len", (p.B,), torch.int32, device)
    if key_mask is not None:
        if key_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"key_mask: {key_mask.dtype}, expected torch.bool or torch.uint8")
        _want(key_mask, "key_mask", (p.B, p.Nk), key_mask.dtype, device)


def cross_forward(p: CrossProblem, Q, K, V, kv_len=None, key_mask=None, O=None, lse=None, return_lse=False,
                  ws=None, stream=None):
    """Cross attention of Q [B,H,Nq,d] to K, V [B,Hkv,Nk,d] (strided views are fine: rows of d
    contiguous channels, strides of a multiple of 16 bytes).  ``kv_len`` [B] int32: the first
    kv_len[b] keys are attended; ``key_mask`` [B,Nk] bool: the keys that are.  Returns O, or
    (O, lse [B,H,Nq] fp32) with ``return_lse``; a new O has Q's order of dimensions."""
    import torch

    dt, dev = _torch_dtype(p.dtype), Q.device
    qs, ks = p._shapes
    sq = _rows(Q, "Q", qs, dt, dev)
    sk = _rows(K, "K", ks, dt, dev)
    sv = _rows(V, "V", ks, dt, dev)
    if kv_len is not None or key_mask is not None:
        _cross_masks(p, kv_len, key_mask, dev)
    lib = _lib()
    with _On(dev, stream) as st:
        if O is None:
            O = torch.empty_like(Q)
        so = _rows(O, "O", qs, dt, dev)
        if lse is not None:
            _want(lse, "lse", qs[:3], torch.float32, dev)
        elif return_lse:
            lse = torch.empty(qs[:3], dtype=torch.float32, device=dev)
        c = p._packed(sq, sk, sv, so)
        ws, nbytes = _workspace(ws, dev, lib.la_cross_workspace_bytes, c)
        rc = lib.la_cross_forward(c, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _p(kv_len), _p(key_mask), O.data_ptr(),
                                  _p(lse), ws.data_ptr(), nbytes, st)
    if rc:
        raise LaError(rc, "la_cross_forward")
    return (O, lse) if return_lse else O


def cross_backward(p: CrossProblem, Q, K, V, O, lse, dO, kv_len=None, key_mask=None, grads=None, ws=None, stream=None):
    """Gradients (dQ, dK, dV) of ``cross_forward`` given its O and lse and the output gradient dO."""
    import torch

    dt, dev = _torch_dtype(p.dtype), Q.device
    qs, ks = p._shapes
    sq = _rows(Q, "Q", qs, dt, dev)
    sk = _rows(K, "K", ks, dt, dev)
    sv = _rows(V, "V", ks, dt, dev)
    so = _rows(O, "O", qs, dt, dev)
    sg = _rows(dO, "dO", qs, dt, dev)
    _want(lse, "lse", qs[:3], torch.float32, dev)
    if kv_len is not None or key_mask is not None:
        _cross_masks(p, kv_len, key_mask, dev)
    lib = _lib()
    with _On(dev, stream) as st:
        dQ, dK, dV = grads if grads is not None else (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V))
        c = p._packed(sq, sk, sv, so, sg, _rows(dQ, "dQ", qs, dt, dev), _rows(dK, "dK", ks, dt, dev),
                      _rows(dV, "dV", ks, dt, dev))
        ws, nbytes = _workspace(ws, dev, lib.la_cross_workspace_bytes, c)
        rc = lib.la_cross_backward(c, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _p(kv_len), _p(key_mask), O.data_ptr(),
                                   lse.data_ptr(), dO.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
                                   ws.data_ptr(), nbytes, st)
    if rc:
        raise LaError(rc, "la_cross_backward")
    return dQ, dK, dV


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

    def _packed(self, sx: int, sy: int, sdy: int, sdx: int) -> bytes:
        return _NORM(self.rows, self.cols, self.groups, sx, sy, sdy, sdx, self.eps,
                     LA_BF16 if self.dtype == "bf16" else LA_F32, 0)

    def c(self) -> LaNormProblem:
        """The C struct for dense tensors."""
        return LaNormProblem.from_buffer_copy(self._packed(self.cols, self.cols, self.cols, self.cols))


_NORM = struct.Struct("=7qfiI4x").pack


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


def _param(t, name, p: NormProblem, dev):
    import torch

    if t is not None:
        shape = (p.cols,) if t.dim() == 1 and p.groups == 1 else (p.groups, p.cols)
        _want(t, name, shape, torch.float32, dev)


def layernorm_forward(p: NormProblem, x, weight=None, bias=None, y=None, mean=None, rstd=None, return_stats=False,
                      stream=None):
    """y = (x - mean) rstd weight_g + bias_g over the rows of x [rows, cols] (row strides are fine).
    ``weight``, ``bias``: fp32 [groups, cols] ([cols] with one group) or None.  ``y`` may be ``x``.
    Returns y, or (y, mean, rstd) ([rows] fp32) with ``return_stats``."""
    import torch

    dev, dt, shape = x.device, _torch_dtype(p.dtype), (p.rows, p.cols)
    sx = _rows(x, "x", shape, dt, dev)
    _param(weight, "weight", p, dev)
    _param(bias, "bias", p, dev)
    lib = _lib()
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty(shape, dtype=dt, device=dev)
        sy = _rows(y, "y", shape, dt, dev)
        for t, name in ((mean, "mean"), (rstd, "rstd")):
            if t is not None:
                _want(t, name, (p.rows,), torch.float32, dev)
        if return_stats or mean is not None or rstd is not None:
            mean = torch.empty(p.rows, dtype=torch.float32, device=dev) if mean is None else mean
            rstd = torch.empty(p.rows, dtype=torch.float32, device=dev) if rstd is None else rstd
        rc = lib.la_layernorm_forward(p._packed(sx[0], sy[0], 0, 0), x.data_ptr(), _p(weight), _p(bias), y.data_ptr(),
                                      _p(mean), _p(rstd), st)
    if rc:
        raise LaError(rc, "la_layernorm_forward")
    return (y, mean, rstd) if return_stats else y


def layernorm_backward(p: NormProblem, x, dy, mean, rstd, weight=None, dx=None, dweight=None, dbias=None,
                       param_grads=True, ws=None, stream=None):
    """(dx, dweight, dbias) of ``layernorm_forward``; dweight and dbias are fp32 [groups, cols], or
    None with ``param_grads`` False (then only those given are computed).  ``dx`` may be ``dy``."""
    import torch

    dev, dt, shape = x.device, _torch_dtype(p.dtype), (p.rows, p.cols)
    sx = _rows(x, "x", shape, dt, dev)
    sdy = _rows(dy, "dy", shape, dt, dev)
    _want(mean, "mean", (p.rows,), torch.float32, dev)
    _want(rstd, "rstd", (p.rows,), torch.float32, dev)
    for t, name in ((weight, "weight"), (dweight, "dweight"), (dbias, "dbias")):
        _param(t, name, p, dev)
    lib = _lib()
    with _On(dev, stream) as st:
        if dx is None:
            dx = torch.empty(shape, dtype=dt, device=dev)
        sdx = _rows(dx, "dx", shape, dt, dev)
        if param_grads:
            gs = (p.groups, p.cols)
            dweight = torch.empty(gs, dtype=torch.float32, device=dev) if dweight is None else dweight
            dbias = torch.empty(gs, dtype=torch.float32, device=dev) if dbias is None else dbias
        c = p._packed(sx[0], 0, sdy[0], sdx[0])
        ws, nbytes = _workspace(ws, dev, lib.la_layernorm_workspace_bytes, p._packed(p.cols, p.cols, p.cols, p.cols))
        rc = lib.la_layernorm_backward(c, x.data_ptr(), dy.data_ptr(), _p(weight), mean.data_ptr(), rstd.data_ptr(),
                                       dx.data_ptr(), _p(dweight), _p(dbias), ws.data_ptr(), nbytes, st)
    if rc:
        raise LaError(rc, "la_layernorm_backward")
    return dx, dweight, dbias


# ------------------------------------------------------------------------------- gradient clipping
def _norm_call(tensors, max_norm, out, norm, ws, stream):
    import torch

    lib = _lib()
    arr, index = _lists().grad_list(list(tensors), None if out is None else list(out))
    n = len(arr) // ctypes.sizeof(LaGrad)
    if n:
        dev = torch.device("cuda", index)
    else:
        dev = norm.device if norm is not None else torch.device("cuda", torch.cuda.current_device())
    with _On(dev, stream) as st:
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=dev)
        elif norm.numel() != 1 or norm.dtype is not torch.float32 or norm.device != dev:
            raise ValueError(f"norm: one fp32 element on {dev} is expected")
        ws, nbytes = _workspace(ws, dev, lib.la_clip_workspace_bytes, n)
        if max_norm is None:
            rc = lib.la_grad_norm(arr, n, norm.data_ptr(), ws.data_ptr(), nbytes, st)
        else:
            rc = lib.la_clip_grad_norm(arr, n, float(max_norm), norm.data_ptr(), ws.data_ptr(), nbytes, st)
    if rc:
        raise LaError(rc, "la_grad_norm" if max_norm is None else "la_clip_grad_norm")
    return norm


def grad_norm(tensors, norm=None, ws=None, stream=None):
    """The 2-norm over all elements of a list of contiguous bf16 / fp32 tensors, as a fp32 scalar
    tensor (``norm`` if given)."""
    return _norm_call(tensors, None, None, norm, ws, stream)


def clip_grad_norm(tensors, max_norm, out=None, norm=None, ws=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of
    ``out``, and returns their norm before that.  Nothing is copied to the host."""
    if max_norm is None:
        raise ValueError("max_norm: a number is expected")
    return _norm_call(tensors, max_norm, out, norm, ws, stream)
