"""Operators of the block around the token mixer, and of its training step: cross attention to an
encoder's states, layer norm, and the global gradient norm with clipping (the ``la_cross_*``,
``la_layernorm_*`` and ``la_*grad_norm`` entry points of include/la.h).

As in ``binding.py``, every step runs in the CUDA library; this module checks shapes, types and
devices (``ValueError``), reads strides and passes pointers.  The library's own checks raise
``LaError``.  Work goes to ``stream``, by default the current stream of the tensors' device; what a
call allocates (outputs that are not given, a workspace that is not given) belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
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
        C, N, G = (ctypes.POINTER(t) for t in (LaCrossProblem, LaNormProblem, LaGrad))
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


def _ok(rc: int, where: str):
    if rc != 0:
        raise LaError(rc, where)


def _torch_dtype(name: str):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


def _want(t, name: str, shape, dtype, device, dense: bool = False):
    """Raises ValueError unless ``t`` is a CUDA tensor of this shape, type and device."""
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, expected {device} (a CUDA device)")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _out(t, name: str, shape, dtype, device, dense: bool = False):
    """``t`` checked, or a new tensor."""
    import torch

    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, shape, dtype, device, dense)
    return t


@contextlib.contextmanager
def _on(device, stream):
    """Makes ``device`` and ``stream`` current, so that the library's device queries and the
    caching allocator see them; gives the stream's handle."""
    import torch

    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream
    elif torch.cuda.current_device() == device.index:
        yield torch.cuda.current_stream().cuda_stream
    else:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream().cuda_stream


def _workspace(ws, device, nbytes):
    """(tensor, size): the given workspace, or a new one of ``nbytes()`` bytes."""
    import torch

    if ws is None:
        n = nbytes()
        return torch.empty(max(n, 16), dtype=torch.uint8, device=device), n
    if isinstance(ws, tuple):  # what cross_workspace() and its like return
        ws = ws[0]
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

    def c(self, **tensors) -> LaCrossProblem:
        """The C struct; a tensor that is not given counts as dense."""
        scale = self.d ** -0.5 if self.scale is None else self.scale
        c = LaCrossProblem(self.B, self.H, self.kv_heads, self.Nq, self.Nk, self.d,
                           LA_BF16 if self.dtype == "bf16" else LA_F32, float(scale),
                           LA_FLAG_FORCE_SIMT if self.force_simt else 0)
        for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
            t = tensors.get(name)
            if t is None:
                keys = name in ("k", "v", "dk", "dv")
                n = self.Nk if keys else self.Nq
                s = ((self.kv_heads if keys else self.H) * n * self.d, n * self.d, self.d)
            else:
                s = t.stride()
            setattr(c, name, LaStrides(*s[:3]))
        return c


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


def _rows(t, name, shape, dtype, device):
    _want(t, name, shape, dtype, device)
    if t.numel() and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")


def _cross_masks(p: CrossProblem, kv_len, key_mask, device):
    import torch

    if kv_len is not None:
        _want(kv_len, "kv_len", (p.B,), torch.int32, device, dense=True)
    if key_mask is not None:
        if key_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"key_mask: {key_mask.dtype}, expected torch.bool or torch.uint8")
        _want(key_mask, "key_mask", (p.B, p.Nk), key_mask.dtype, device, dense=True)


def cross_forward(p: CrossProblem, Q, K, V, kv_len=None, key_mask=None, O=None, lse=None, return_lse=False,
                  ws=None, stream=None):
    """Cross attention of Q [B,H,Nq,d] to K, V [B,Hkv,Nk,d] (strided views are fine: rows of d
    contiguous channels, strides of a multiple of 16 bytes).  ``kv_len`` [B] int32: the first
    kv_len[b] keys are attended; ``key_mask`` [B,Nk] bool: the keys that are.  Returns O, or
    (O, lse [B,H,Nq] fp32) with ``return_lse``; a new O has Q's order of dimensions."""
    import torch

    dt, dev = _torch_dtype(p.dtype), Q.device
    qs, ks = (p.B, p.H, p.Nq, p.d), (p.B, p.kv_heads, p.Nk, p.d)
    _rows(Q, "Q", qs, dt, dev)
    _rows(K, "K", ks, dt, dev)
    _rows(V, "V", ks, dt, dev)
    _cross_masks(p, kv_len, key_mask, dev)
    with _on(dev, stream) as st:
        if O is None:
            O = torch.empty_like(Q)
        _rows(O, "O", qs, dt, dev)
        if lse is not None or return_lse:
            lse = _out(lse, "lse", qs[:3], torch.float32, dev, dense=True)
        c = p.c(q=Q, k=K, v=V, o=O)
        lib = _lib()
        ws, nbytes = _workspace(ws, dev, lambda: lib.la_cross_workspace_bytes(ctypes.byref(c)))
        _ok(lib.la_cross_forward(ctypes.byref(c), _p(Q), _p(K), _p(V), _p(kv_len), _p(key_mask), _p(O), _p(lse),
                                 _p(ws), nbytes, st), "la_cross_forward")
    return (O, lse) if return_lse else O


def cross_backward(p: CrossProblem, Q, K, V, O, lse, dO, kv_len=None, key_mask=None, grads=None, ws=None, stream=None):
    """Gradients (dQ, dK, dV) of ``cross_forward`` given its O and lse and the output gradient dO."""
    import torch

    dt, dev = _torch_dtype(p.dtype), Q.device
    qs, ks = (p.B, p.H, p.Nq, p.d), (p.B, p.kv_heads, p.Nk, p.d)
    for t, name, shape in ((Q, "Q", qs), (K, "K", ks), (V, "V", ks), (O, "O", qs), (dO, "dO", qs)):
        _rows(t, name, shape, dt, dev)
    _want(lse, "lse", qs[:3], torch.float32, dev, dense=True)
    _cross_masks(p, kv_len, key_mask, dev)
    with _on(dev, stream) as st:
        dQ, dK, dV = grads if grads is not None else (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V))
        for t, name, shape in ((dQ, "dQ", qs), (dK, "dK", ks), (dV, "dV", ks)):
            _rows(t, name, shape, dt, dev)
        c = p.c(q=Q, k=K, v=V, o=O, dout=dO, dq=dQ, dk=dK, dv=dV)
        lib = _lib()
        ws, nbytes = _workspace(ws, dev, lambda: lib.la_cross_workspace_bytes(ctypes.byref(c)))
        _ok(lib.la_cross_backward(ctypes.byref(c), _p(Q), _p(K), _p(V), _p(kv_len), _p(key_mask), _p(O), _p(lse),
                                  _p(dO), _p(dQ), _p(dK), _p(dV), _p(ws), nbytes, st), "la_cross_backward")
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

    def c(self, x=None, y=None, dy=None, dx=None) -> LaNormProblem:
        s = [self.cols if t is None else t.stride(0) for t in (x, y, dy, dx)]
        return LaNormProblem(self.rows, self.cols, self.groups, *s, float(self.eps),
                             LA_BF16 if self.dtype == "bf16" else LA_F32, 0)


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


def _cols(t, name, p: NormProblem, dev):
    _want(t, name, (p.rows, p.cols), _torch_dtype(p.dtype), dev)
    if t.numel() and p.cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous")


def _param(t, name, p: NormProblem, dev):
    import torch

    if t is not None:
        if t.dim() == 1 and p.groups == 1:
            t = t[None]
        _want(t, name, (p.groups, p.cols), torch.float32, dev, dense=True)


def layernorm_forward(p: NormProblem, x, weight=None, bias=None, y=None, mean=None, rstd=None, return_stats=False,
                      stream=None):
    """y = (x - mean) rstd weight_g + bias_g over the rows of x [rows, cols] (row strides are fine).
    ``weight``, ``bias``: fp32 [groups, cols] ([cols] with one group) or None.  ``y`` may be ``x``.
    Returns y, or (y, mean, rstd) ([rows] fp32) with ``return_stats``."""
    import torch

    dev = x.device
    _cols(x, "x", p, dev)
    _param(weight, "weight", p, dev)
    _param(bias, "bias", p, dev)
    with _on(dev, stream) as st:
        if y is None:
            y = torch.empty((p.rows, p.cols), dtype=x.dtype, device=dev)
        _cols(y, "y", p, dev)
        if return_stats or mean is not None or rstd is not None:
            mean = _out(mean, "mean", (p.rows,), torch.float32, dev, dense=True)
            rstd = _out(rstd, "rstd", (p.rows,), torch.float32, dev, dense=True)
        c = p.c(x=x, y=y)
        _ok(_lib().la_layernorm_forward(ctypes.byref(c), _p(x), _p(weight), _p(bias), _p(y), _p(mean), _p(rstd), st),
            "la_layernorm_forward")
    return (y, mean, rstd) if return_stats else y


def layernorm_backward(p: NormProblem, x, dy, mean, rstd, weight=None, dx=None, dweight=None, dbias=None,
                       param_grads=True, ws=None, stream=None):
    """(dx, dweight, dbias) of ``layernorm_forward``; dweight and dbias are fp32 [groups, cols], or
    None with ``param_grads`` False (then only those given are computed).  ``dx`` may be ``dy``."""
    import torch

    dev = x.device
    _cols(x, "x", p, dev)
    _cols(dy, "dy", p, dev)
    _param(weight, "weight", p, dev)
    _want(mean, "mean", (p.rows,), torch.float32, dev, dense=True)
    _want(rstd, "rstd", (p.rows,), torch.float32, dev, dense=True)
    with _on(dev, stream) as st:
        if dx is None:
            dx = torch.empty((p.rows, p.cols), dtype=x.dtype, device=dev)
        _cols(dx, "dx", p, dev)
        for t, name in ((dweight, "dweight"), (dbias, "dbias")):
            _param(t, name, p, dev)
        if param_grads:
            shape = (p.groups, p.cols)
            dweight = torch.empty(shape, dtype=torch.float32, device=dev) if dweight is None else dweight
            dbias = torch.empty(shape, dtype=torch.float32, device=dev) if dbias is None else dbias
        c = p.c(x=x, dy=dy, dx=dx)
        lib = _lib()
        ws, nbytes = _workspace(ws, dev, lambda: lib.la_layernorm_workspace_bytes(ctypes.byref(c)))
        _ok(lib.la_layernorm_backward(ctypes.byref(c), _p(x), _p(dy), _p(weight), _p(mean), _p(rstd), _p(dx),
                                      _p(dweight), _p(dbias), _p(ws), nbytes, st), "la_layernorm_backward")
    return dx, dweight, dbias


# ------------------------------------------------------------------------------- gradient clipping
def _grad_list(tensors, out):
    import torch

    n = len(tensors)
    if out is not None and len(out) != n:
        raise ValueError(f"out: {len(out)} tensors for {n} gradients")
    kinds = {torch.bfloat16: LA_BF16, torch.float32: LA_F32}
    arr = (LaGrad * max(n, 1))()
    dev = tensors[0].device if n else None
    for i, t in enumerate(tensors):
        o = t if out is None else out[i]
        kind = kinds.get(t.dtype)
        if kind is None:
            raise ValueError(f"gradient {i}: {t.dtype}, expected torch.bfloat16 or torch.float32")
        if t.device != dev or dev.type != "cuda":
            raise ValueError(f"gradient {i}: on {t.device}, expected {dev} (a CUDA device)")
        if not t.is_contiguous():
            raise ValueError(f"gradient {i}: must be contiguous")
        if o is not t and (o.dtype is not t.dtype or o.device != dev or o.shape != t.shape or not o.is_contiguous()):
            raise ValueError(f"out {i}: must be a contiguous tensor like its gradient")
        g = arr[i]
        g.in_, g.out, g.numel, g.dtype = t.data_ptr(), o.data_ptr(), t.numel(), kind
    return arr, n, dev


def _norm_call(tensors, max_norm, out, norm, ws, stream):
    import torch

    tensors = list(tensors)
    arr, n, dev = _grad_list(tensors, out)
    if dev is None:
        dev = norm.device if norm is not None else torch.device("cuda", torch.cuda.current_device())
    with _on(dev, stream) as st:
        norm = _out(norm, "norm", (), torch.float32, dev)
        lib = _lib()
        ws, nbytes = _workspace(ws, dev, lambda: lib.la_clip_workspace_bytes(n))
        if max_norm is None:
            _ok(lib.la_grad_norm(arr, n, _p(norm), _p(ws), nbytes, st), "la_grad_norm")
        else:
            _ok(lib.la_clip_grad_norm(arr, n, float(max_norm), _p(norm), _p(ws), nbytes, st), "la_clip_grad_norm")
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
