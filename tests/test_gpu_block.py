"""The operators of the block around the token mixer, on the GPU, against fp64: cross attention,
layer norm, gradient norm and clipping.  Tolerances are those that oracle/block_oracle.py derives
from the roundings of each type."""
import math

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P_UNIT = 2.0 ** -8  # probabilities (and dS) as bf16 matrix operands


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(shape, dtype, g, layout="bhnd"):
    if layout == "bnhd":
        B, H, N, d = shape
        return torch.randn((B, N, H, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        over = torch.where(same, 0.0, (got - want).abs() / tol)
        at = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(over.max()):.2f} x the "
                             f"bound; first at {at}: got {float(got[tuple(at)])}, want {float(want[tuple(at)])}")


def unit(dtype, simt):
    return P_UNIT if dtype == "bf16" and not simt else 0.0


def inputs(B, H, Hkv, Nq, Nk, d, dtype, pad, layout="bhnd", seed=0):
    g = gen(seed)
    Q = rnd((B, H, Nq, d), DT[dtype], g, layout)
    if layout == "bnhd":
        kv = torch.randn((B, Nk, 2, Hkv, d), generator=g, device="cuda").to(DT[dtype])
        K, V = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    else:
        K, V = rnd((B, Hkv, Nk, d), DT[dtype], g), rnd((B, Hkv, Nk, d), DT[dtype], g)
    kv_len = key_mask = None
    if pad in ("len", "both"):  # 0, all, and what lies between; values outside [0, Nk] are clamped
        kv_len = torch.tensor([[Nk, 0, Nk // 2 + 1, Nk + 5, -3][(b + seed) % 5] for b in range(B)],
                              dtype=torch.int32, device="cuda")
    if pad in ("mask", "both"):
        key_mask = torch.rand((B, Nk), generator=g, device="cuda") < 0.6
        if B > 1:
            key_mask[1] = False
    ok = bo.attended(B, Nk, kv_len, key_mask, "cuda")
    for t, bad in ((K, math.nan), (V, math.inf)):  # what unattended rows hold has no influence
        hole = ~ok[:, None, :, None].expand(B, Hkv, Nk, d)
        t.masked_fill_(hole, bad)
        t.masked_fill_(hole & (torch.arange(Nk, device="cuda") % 2 == 0)[None, None, :, None], torch.finfo(t.dtype).min)
    return Q, K, V, kv_len, key_mask, ok


# (B, H, Hkv, Nq, Nk, d)
SHAPES = [
    (1, 1, 1, 1, 1, 128), (2, 3, 3, 1, 65, 64), (1, 2, 1, 5, 0, 32), (2, 2, 2, 64, 64, 128), (3, 4, 2, 129, 127, 128),
    (1, 6, 3, 300, 129, 64), (2, 2, 1, 257, 300, 128), (1, 2, 2, 255, 513, 32), (5, 4, 1, 1, 700, 128),
    (1, 1, 1, 2, 4099, 64), (1, 2, 2, 1025, 16, 128), (2, 8, 2, 33, 1000, 128), (1, 3, 1, 700, 260, 64),
]


@pytest.mark.parametrize("pad", ["none", "len", "mask", "both"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,simt", [("f32", False), ("bf16", True), ("bf16", False)])
def test_cross_forward(shape, dtype, simt, pad):
    B, H, Hkv, Nq, Nk, d = shape
    layout = "bnhd" if (Nq + Nk) % 2 else "bhnd"
    Q, K, V, kv_len, key_mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, pad, layout)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype, force_simt=simt)
    O, lse = la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=key_mask, return_lse=True)
    assert O.stride() == torch.empty_like(Q).stride()
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok, unit(dtype, simt))
    close(O, o, to, "O")
    close(lse, l, tl, "lse")
    again = la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=key_mask)
    assert torch.equal(O, again)
    assert la.device_error() == 0


@pytest.mark.parametrize("pad", ["none", "len", "mask", "both"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,simt", [("f32", False), ("bf16", True), ("bf16", False)])
def test_cross_backward(shape, dtype, simt, pad):
    B, H, Hkv, Nq, Nk, d = shape
    layout = "bnhd" if (Nq + Nk) % 2 else "bhnd"
    Q, K, V, kv_len, key_mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, pad, layout, seed=1)
    dO = rnd((B, H, Nq, d), DT[dtype], gen(5), "bnhd" if Nk % 2 else "bhnd")
    o, l, _, _ = bo.cross_forward(Q, K, V, d ** -0.5, ok)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype, force_simt=simt)
    args = (Q, K, V, o.to(DT[dtype]), l.float(), dO)
    got = la.cross_backward(p, *args, kv_len=kv_len, key_mask=key_mask)
    want, tol = bo.cross_backward(Q, K, V, dO, d ** -0.5, ok, unit(dtype, simt))
    for a, b, t, n in zip(got, want, tol, ("dQ", "dK", "dV")):
        close(a, b, t, n)
    again = la.cross_backward(p, *args, kv_len=kv_len, key_mask=key_mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert la.device_error() == 0


def test_cross_scores_of_any_size():
    # large scores of both signs: the running maximum moves late, and far
    B, H, Nq, Nk, d = 1, 2, 200, 400, 64
    g = gen(3)
    for dtype in ("f32", "bf16"):
        Q, K, V = (rnd((B, H, n, d), DT[dtype], g) for n in (Nq, Nk, Nk))
        K = K * torch.linspace(-30, 30, Nk, device="cuda")[None, None, :, None].to(DT[dtype])
        ok = bo.attended(B, Nk, device="cuda")
        p = la.CrossProblem(B=B, H=H, Nq=Nq, Nk=Nk, d=d, dtype=dtype, scale=0.5)
        O, lse = la.cross_forward(p, Q, K, V, return_lse=True)
        o, l, to, tl = bo.cross_forward(Q, K, V, 0.5, ok, unit(dtype, False))
        close(O, o, to, "O")
        close(lse, l, tl, "lse")


# (rows, cols, groups)
NORMS = [(1, 1, 1), (3, 1001, 1), (5, 8, 5), (37, 256, 1), (64, 512, 2), (130, 520, 1), (9, 1000, 3), (300, 2048, 1),
         (21, 4096, 3), (7, 4104, 1), (6, 8192, 2), (4, 16384, 1), (5, 8191, 1), (3, 16383, 1), (2000, 100, 4), (700, 33, 1)]


@pytest.mark.parametrize("affine", ["both", "none", "weight"])
@pytest.mark.parametrize("shape", NORMS, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm(dtype, shape, affine):
    rows, cols, groups = shape
    g = gen(rows)
    x = (torch.randn((rows, cols), generator=g, device="cuda") * 1.5 + 4.0).to(DT[dtype])
    w = 1 + 0.2 * torch.randn((groups, cols), generator=g, device="cuda") if affine != "none" else None
    b = torch.randn((groups, cols), generator=g, device="cuda") if affine == "both" else None
    p = la.NormProblem(rows=rows, cols=cols, groups=groups, dtype=dtype)
    got = la.layernorm_forward(p, x, w, b, return_stats=True)
    want, tol = bo.norm_forward(x, w, b, p.eps)
    for a, r, t, n in zip(got, want, tol, ("y", "mean", "rstd")):
        close(a, r, t, n)
    dy = torch.randn((rows, cols), generator=g, device="cuda").to(DT[dtype])
    mean, rstd = got[1], got[2]
    grads = la.layernorm_backward(p, x, dy, mean, rstd, w)
    want, tol = bo.norm_backward(x, dy, w, mean, rstd, groups)
    for a, r, t, n in zip(grads, want, tol, ("dx", "dweight", "dbias")):
        close(a, r, t, n)
    again = la.layernorm_backward(p, x, dy, mean, rstd, w)
    assert all(torch.equal(a, c) for a, c in zip(grads, again))


@pytest.mark.parametrize("cols", [136, 33, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_strides_and_in_place(dtype, cols):
    rows, p = 19, la.NormProblem(rows=19, cols=cols, dtype=dtype)
    g = gen(2)
    buf = torch.randn((rows, 2 * cols + 8), generator=g, device="cuda").to(DT[dtype])
    x, y = buf[:, :cols], buf[:, cols:2 * cols]
    keep = buf[:, 2 * cols:].clone()
    want, tol = bo.norm_forward(x.clone(), None, None, p.eps)
    _, mean, rstd = la.layernorm_forward(p, x, y=y, return_stats=True)  # side by side in one buffer
    close(y, want[0], tol[0], "y")
    dense = la.layernorm_forward(p, x.contiguous())
    dy = torch.randn((rows, cols), generator=g, device="cuda").to(DT[dtype])
    want, tol = bo.norm_backward(x, dy, None, mean, rstd, 1)
    dx, dw, _ = la.layernorm_backward(p, x, dy, mean, rstd, dx=dy)
    assert dx is dy
    close(dx, want[0], tol[0], "dx over dy")
    close(dw, want[1], tol[1], "dweight")
    assert la.layernorm_forward(p, x, y=x) is x
    assert torch.equal(x, dense) and torch.equal(buf[:, 2 * cols:], keep)
    with pytest.raises(la.LaError, match="LA_ERR_SHAPE"):
        la.layernorm_forward(p, x, y=buf[:, 4:cols + 4])
    with pytest.raises(la.LaError, match="LA_ERR_SHAPE"):
        la.layernorm_backward(p, x, buf[:, cols:2 * cols], mean, rstd, dx=buf[:, cols - 4:2 * cols - 4])


def test_layernorm_without_rows_or_parameter_gradients():
    p = la.NormProblem(rows=0, cols=24, groups=3)
    x = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = la.layernorm_forward(p, x, return_stats=True)
    dx, dw, db = la.layernorm_backward(p, x, x, mean, rstd)
    assert y.shape == dx.shape == (0, 24) and not dw.any() and not db.any()
    p = la.NormProblem(rows=50, cols=24)
    x = torch.randn((50, 24), device="cuda").to(torch.bfloat16)
    _, mean, rstd = la.layernorm_forward(p, x, return_stats=True)
    dx, dw, db = la.layernorm_backward(p, x, x, mean, rstd, param_grads=False)
    full = la.layernorm_backward(p, x, x, mean, rstd)
    only = la.layernorm_backward(p, x, x, mean, rstd, param_grads=False, dbias=torch.empty(24, device="cuda"))
    assert dw is None and db is None and torch.equal(dx, full[0])
    assert only[1] is None and torch.equal(only[2], full[2][0])


SIZES = [[1], [0], [], [5, 0, 16384, 16385, 7, 100003], [64 * i % 1001 + 1 for i in range(1100)], [3 << 20, 17]]


@pytest.mark.parametrize("sizes", SIZES, ids=len)
@pytest.mark.parametrize("place", ["in", "out"])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip_grad_norm(sizes, place, shift):
    g = gen(len(sizes))
    base = [torch.randn(n + shift, generator=g, device="cuda").to(torch.float32 if i % 3 == 1 else torch.bfloat16)
            for i, n in enumerate(sizes)]
    grads = [b[shift:] for b in base]  # with a shift of 1, aligned to their type only
    ref = bo.grad_norm(grads)
    assert abs(float(la.grad_norm(grads)) - ref) <= 4 * bo.U32 * ref
    for max_norm in (0.25 * ref if ref else 1.0, 2.0 * ref + 1.0):
        src = [t.clone() for t in base]
        src = [t[shift:] for t in src]
        outs = [torch.full_like(t, 7.0) for t in base]
        outs = [t[shift:] for t in outs] if place == "out" else None
        norm = la.clip_grad_norm(src, max_norm, out=outs)
        assert abs(float(norm) - ref) <= 4 * bo.U32 * ref
        c = min(1.0, max_norm / (ref + 1e-6))
        for i, (a, b, t) in enumerate(zip(src, outs or src, grads)):
            want = t.double() * c
            close(b, want, (bo.HALF_STEP[t.dtype] + 6 * bo.U32) * want.abs(), f"gradient {i}")
            if outs is not None:
                assert torch.equal(a, t)


def test_grad_norm_range():
    for dtype in (torch.bfloat16, torch.float32):
        for scale in (1e30, 3e37, 1e-30, 1e-38, 1e-20):
            t = (torch.randn(40001, generator=gen(1), device="cuda") * scale).to(dtype)
            parts = [t[:1001], torch.zeros(50, dtype=dtype, device="cuda"), t[1001:]]
            # the norm is handed out in fp32: above its range (sqrt(40001) * 3e37 is) it is infinite
            ref = float(torch.tensor(bo.grad_norm(parts), dtype=torch.float64).float())
            got = float(la.grad_norm(parts))
            # the norm itself may be below fp32's normal range, where a step is 2^-149
            assert got == ref or abs(got - ref) <= 4 * bo.U32 * ref + 2.0 ** -149, (dtype, scale, got, ref)
    t = torch.ones(100, device="cuda")
    t[50] = math.inf
    assert float(la.clip_grad_norm([t], 1.0)) == math.inf
    assert t[50].isnan() and not t[:50].any()
    t = torch.ones(100, device="cuda")
    t[3] = math.nan
    assert math.isnan(float(la.clip_grad_norm([t], 1.0))) and t.isnan().all()


def test_clip_refuses_overlaps():
    t = torch.ones(64, device="cuda")
    for grads, out in (([t, t], None), ([t[:40], t[30:]], None), ([t[:32]], [t[16:48]]),
                       ([t[:32], t[32:]], [t[32:], torch.ones(32, device="cuda")])):
        with pytest.raises(la.LaError, match="LA_ERR_SHAPE"):
            la.clip_grad_norm(grads, 1.0, out=out)
    assert float(la.grad_norm([t, t])) == pytest.approx(math.sqrt(128), rel=1e-6)  # reading twice is no overlap
    la.clip_grad_norm([t[:32], t[:32]], 1.0, out=[torch.empty(32, device="cuda"), torch.empty(32, device="cuda")])


# (B, H, Hkv, Nq, Nk, d): several key tiles; the keys split; a few rows, split and not
SPECIAL = [(2, 2, 2, 140, 300, 64), (1, 1, 1, 130, 2100, 128), (1, 4, 2, 1, 700, 128), (2, 2, 1, 3, 40, 32)]
PATHS = [("f32", False), ("bf16", True), ("bf16", False)]


@pytest.mark.parametrize("shape", SPECIAL, ids=str)
@pytest.mark.parametrize("dtype,simt", PATHS)
def test_cross_forward_scores_of_minus_infinity(shape, dtype, simt):
    """A score of -inf weighs 0, also where a whole tile has nothing else; a row of them has o = 0."""
    B, H, Hkv, Nq, Nk, d = shape
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype, force_simt=simt)
    Q, K, V, *_, ok = inputs(*shape, dtype, "none", seed=2)
    Q[..., 0] = Q[..., 0].abs() + 0.5
    gone = Nk * 2 // 3
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok & (torch.arange(Nk, device="cuda") >= gone), unit(dtype, simt))
    K[:, :, :gone, 0] = -math.inf
    O, lse = la.cross_forward(p, Q, K, V, return_lse=True)
    close(O, o, to, "O")
    close(lse, l, tl, "lse")
    K[..., 0] = -math.inf
    O, lse = la.cross_forward(p, Q, K, V, return_lse=True)
    assert not O.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("shape", SPECIAL, ids=str)
@pytest.mark.parametrize("dtype,simt", PATHS)
def test_cross_forward_hands_nan_on(shape, dtype, simt):
    """NaN that is attended comes out as NaN where it belongs, and nowhere else."""
    B, H, Hkv, Nq, Nk, d = shape
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype, force_simt=simt)
    Q, K, V, *_ = inputs(*shape, dtype, "none", seed=3)
    whole, l0 = la.cross_forward(p, Q, K, V, return_lse=True)
    heads = slice((Hkv - 1) * (H // Hkv), H)  # those that read the last key head

    def check(q, k, v, at, channels=slice(None), lse_too=True):
        O, lse = la.cross_forward(p, q, k, v, return_lse=True)
        hit = torch.zeros(O.shape, dtype=torch.bool, device="cuda")
        hit[at][..., channels] = True
        assert O[hit].isnan().all() and torch.equal(O[~hit], whole[~hit])
        rows = hit.any(3) if lse_too else torch.zeros_like(l0, dtype=torch.bool)
        assert lse[rows].isnan().all() and torch.equal(lse[~rows], l0[~rows])

    q, k, v, bad = Q.clone(), K.clone(), V.clone(), K.clone()
    q[-1, -1, Nq - 1, 3] = math.nan
    check(q, K, V, (slice(B - 1, B), slice(H - 1, H), slice(Nq - 1, Nq)))
    k[-1, -1, Nk - 1, 5] = math.nan
    check(Q, k, V, (slice(B - 1, B), heads))
    bad[-1, -1] = math.nan
    check(Q, bad, V, (slice(B - 1, B), heads))
    v[-1, -1, Nk // 2, 7] = math.nan
    check(Q, K, v, (slice(B - 1, B), heads), slice(7, 8), lse_too=False)
