"""Plain fp64 definitions of the operators of the block around the token mixer (torch tensors of
any type in, fp64 out, on the tensors' device), and bounds on what rounding may change.

Test infrastructure: nothing here is used by, or shares code with, the CUDA library.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24                                   # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
EXP_U = 2.0 ** -21                                 # an exponential (2 ulp and the rounding of its argument's product)


def attended(B, Nk, kv_len=None, key_mask=None, device="cpu"):
    """[B, Nk] truth values: the keys each batch row attends."""
    ok = torch.ones((B, Nk), dtype=torch.bool, device=device)
    if kv_len is not None:
        ok &= torch.arange(Nk, device=device)[None] < kv_len.to(device).clamp(0, Nk)[:, None]
    if key_mask is not None:
        ok &= key_mask.to(device) != 0
    return ok


def _expand(x, H):
    """[B,Hkv,N,d] -> [B,H,N,d] fp64: head h reads key head h // (H // Hkv)."""
    return x.double().repeat_interleave(H // x.shape[1], dim=1)


def _cross_parts(Q, K, V, scale, ok):
    H = Q.shape[1]
    at = ok[:, None, :, None]
    q, k, v = Q.double(), _expand(K, H).where(at, 0.0), _expand(V, H).where(at, 0.0)
    s = (q @ k.transpose(2, 3)) * scale
    s = s.where(ok[:, None, None, :], -math.inf)
    lse = torch.logsumexp(s, 3)
    p = torch.exp(s - lse[..., None].nan_to_num(neginf=0.0))
    # rounding of a score in fp32: d products and sums, and the scale
    ds = (Q.shape[3] + 4) * U32 * scale * (q.abs() @ k.abs().transpose(2, 3))
    ds = ds + 2 * U32 * s.abs().nan_to_num(posinf=0.0)
    return q, k, v, p, lse, ds


def cross_forward(Q, K, V, scale, ok, p_unit=0.0):
    """(O, lse) in fp64 and the largest allowed difference of each, elementwise: the output's own
    rounding, plus what follows from rounding scores, exponentials and sums in fp32 and the
    probabilities to ``p_unit`` (2^-8 where they are a bf16 matrix operand)."""
    _, _, v, p, lse, ds = _cross_parts(Q, K, V, scale, ok)
    o = p @ v
    n = K.shape[2]
    per = 2 * ds.amax(3, keepdim=True) if n else torch.zeros_like(lse)[..., None]
    per = per + EXP_U + (n + 16) * U32
    tol_o = HALF_STEP[Q.dtype] * o.abs() + 1.01 * (per + p_unit) * (p @ v.abs()) + 1e-30
    tol_l = (per[..., 0] + 4 * U32 * (1 + lse.abs())).nan_to_num(posinf=0.0)
    return o, lse, tol_o, tol_l


def cross_backward(Q, K, V, dO, scale, ok, p_unit=0.0):
    """(dQ, dK, dV) and the largest allowed difference of each, for an O and lse that are the exact
    ones rounded to their types."""
    B, H, Nq, d = Q.shape
    Hkv = K.shape[1]
    q, k, v, p, lse, es = _cross_parts(Q, K, V, scale, ok)
    g = dO.double()
    dp = g @ v.transpose(2, 3)
    D = (p * dp).sum(3, keepdim=True)
    ds = scale * p * (dp - D)
    n = K.shape[2]
    hs = HALF_STEP[Q.dtype]
    # p: the score's rounding, lse's rounding, the exponential
    rel_p = es + EXP_U + 4 * U32 * (1 + lse.abs().nan_to_num(posinf=0.0))[..., None]
    # dp and D: fp32 sums over the channels; O rounded to its type
    e_dp = (d + 4) * U32 * (g.abs() @ v.abs().transpose(2, 3))
    e_D = (hs + (d + 4) * U32) * (g.abs() * (p @ v.abs())).sum(3, keepdim=True)
    e_ds = ds.abs() * (rel_p + p_unit + 4 * U32) + scale * p * (e_dp + e_D)
    e_p = p * (rel_p + p_unit)

    def shared(x):  # sum over the query heads of a key head
        return x.reshape(B, Hkv, H // Hkv, n, d).sum(2)

    rows = Nq * (H // Hkv)
    dq, dk, dv = ds @ k, shared(ds.transpose(2, 3) @ q), shared(p.transpose(2, 3) @ g)
    t_q = hs * dq.abs() + 1.01 * (e_ds @ k.abs()) + (n + 16) * U32 * (ds.abs() @ k.abs()) + 1e-30
    t_k = hs * dk.abs() + 1.01 * shared(e_ds.transpose(2, 3) @ q.abs()) + \
        (rows + 16) * U32 * shared(ds.abs().transpose(2, 3) @ q.abs()) + 1e-30
    t_v = hs * dv.abs() + 1.01 * shared(e_p.transpose(2, 3) @ g.abs()) + \
        (rows + 16) * U32 * shared(p.transpose(2, 3) @ g.abs()) + 1e-30
    return (dq, dk, dv), (t_q, t_k, t_v)


def _per_row(w, rows):
    return w.double().repeat_interleave(rows // w.shape[0], 0)


def norm_forward(x, weight, bias, eps):
    """(y, mean, rstd) and the largest allowed differences; weight, bias: [groups, cols] or None."""
    rows, cols = x.shape
    a = x.double()
    mean = a.mean(1, keepdim=True)
    c = a - mean
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = c * rstd
    w = torch.ones_like(a) if weight is None else _per_row(weight, rows)
    b = torch.zeros_like(a) if bias is None else _per_row(bias, rows)
    y = xh * w + b
    # the mean's rounding moves every value alike; its square enters the variance
    e_mu = (math.log2(cols + 1) + cols / 32 + 4) * U32 * a.abs().mean(1, keepdim=True)
    rel_r = (math.log2(cols + 1) + cols / 32 + 8) * U32 + e_mu ** 2 / (var + eps)
    e_xh = rstd * (e_mu + U32 * (a.abs() + mean.abs())) + xh.abs() * rel_r
    t_y = HALF_STEP[x.dtype] * y.abs() + 1.01 * (e_xh * w.abs() + 4 * U32 * (xh.abs() * w.abs() + b.abs())) + 1e-30
    return (y, mean[:, 0], rstd[:, 0]), (t_y, (e_mu + U32 * mean.abs())[:, 0] + 1e-30, (rstd * (rel_r + 2 * U32))[:, 0])


def norm_backward(x, dy, weight, mean, rstd, groups):
    """(dx, dweight, dbias) from the given statistics, and the largest allowed differences."""
    rows, cols = x.shape
    a, g, r = x.double(), dy.double(), rstd.double()[:, None]
    c = a - mean.double()[:, None]
    xh = c * r
    w = torch.ones_like(a) if weight is None else _per_row(weight, rows)
    gw = g * w
    m1, m2 = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
    dx = r * (gw - m1 - xh * m2)
    e_xh = 3 * U32 * xh.abs() + U32 * c.abs() * r
    n = (math.log2(cols + 1) + cols / 32 + 8) * U32
    e = n * gw.abs().mean(1, keepdim=True) + xh.abs() * (n * (gw * xh).abs().mean(1, keepdim=True) +
                                                        (gw.abs() * e_xh).mean(1, keepdim=True)) + e_xh * m2.abs()
    t_x = HALF_STEP[x.dtype] * dx.abs() + 1.01 * r * (e + 6 * U32 * (gw.abs() + m1.abs() + (xh * m2).abs())) + 1e-30
    per = rows // groups

    def total(t):
        return t.reshape(groups, per, cols).sum(1)

    steps = (per + 16) * U32
    t_w = total((g * xh).abs()) * (steps + 2 * U32) + total(g.abs() * e_xh) + 1e-30
    return (dx, total(g * xh), total(g)), (t_x, t_w, total(g.abs()) * steps + 1e-30)


def grad_norm(tensors):
    """sqrt of the sum of squares, in fp64 (scaled, so that squares stay in range)."""
    top = max([float(t.double().abs().max()) for t in tensors if t.numel()] or [0.0])
    if top == 0.0 or not math.isfinite(top):
        return top
    return top * math.sqrt(sum(float((t.double() / top).square().sum()) for t in tensors))
