"""Host-side checks of the operators of the block around the token mixer (no GPU): the library's
refusals, the binding's, workspace sizes, and the fp64 oracle against finite differences."""
import ctypes

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import block as blk
from oracle import block_oracle as bo

BIG = 1 << 40


def _cross(p, ptrs=(16,) * 3, tail=(None, None, 16, 16), back=False, tweak=None):
    lib = blk._lib()
    c = p.c()
    if tweak:
        tweak(c)
    if back:  # distinct addresses: inputs and outputs may not be the same
        return lib.la_cross_backward(ctypes.byref(c), 16, 32, 48, None, None, 64, 16, 80, 96, 112, 128, 16, 0, None)
    return lib.la_cross_forward(ctypes.byref(c), *ptrs, *tail, 16, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=48), 5), (dict(Nq=-1), 2), (dict(Hkv=3), 2), (dict(Hkv=0), 2), (dict(scale=0.0), 2),
    (dict(scale=float("nan")), 2), (dict(scale=-1.0), 2), (dict(scale=float("inf")), 2),
    (dict(Nq=2 ** 31), 2), (dict(Nk=2 ** 31), 2), (dict(B=2 ** 20, H=2 ** 12), 2),
])
def test_cross_rejects_bad_problems_before_cuda(kw, status):
    args = dict(B=2, H=4, Nq=8, Nk=8, d=64)
    args.update(kw)
    p = la.CrossProblem(**args)
    assert _cross(p) == status
    assert _cross(p, back=True) == status
    assert la.cross_workspace_bytes(p, 148) == 0


def test_cross_rejects_bad_pointers_strides_and_flags_before_cuda():
    p = la.CrossProblem(B=2, H=4, Nq=8, Nk=8, d=64)
    assert _cross(p, (None, 16, 16)) == 1
    assert _cross(p, (16, 24, 32)) == 4
    assert _cross(p, (16, 32, 48), (None, None, None, 16)) == 1
    assert _cross(p, (16, 32, 48), (6, None, 64, 16)) == 4       # kv_len: aligned to its type
    assert _cross(p, (16, 32, 48), (None, None, 16, 16)) == 2    # the output is an input
    for field, index, value, status in (("q", "n", 60, 4), ("q", "n", 0, 2), ("k", "h", -64, 2), ("o", "n", 32, 2),
                                        ("o", "h", 64, 2), ("v", "b", 2 ** 60, 2)):
        assert _cross(p, tweak=lambda c: setattr(getattr(c, field), index, value)) == status, (field, index, value)
    for field in ("dq", "dk", "dv"):
        assert _cross(p, back=True, tweak=lambda c: setattr(getattr(c, field), "n", 32)) == 2
    # strides of extent 1 do not matter
    one = la.CrossProblem(B=1, H=1, Nq=1, Nk=8, d=64)
    assert _cross(one, (None, 16, 16), tweak=lambda c: setattr(c, "q", blk.LaStrides(-1, 3, 0))) == 1
    assert _cross(p, tweak=lambda c: setattr(c, "flags", 2)) == 5
    assert _cross(p, tweak=lambda c: setattr(c, "dtype", 7)) == 5
    lib = blk._lib()
    assert lib.la_cross_forward(None, *([16] * 7), 16, 0, None) == 1


def test_layernorm_rejects_bad_arguments_before_cuda():
    lib = blk._lib()

    def fwd(p, x=16, w=None, b=None, y=1 << 20, mean=None, rstd=None, **fields):
        c = p.c()
        for k, v in fields.items():
            setattr(c, k, v)
        return lib.la_layernorm_forward(ctypes.byref(c), x, w, b, y, mean, rstd, None)

    ok = la.NormProblem(rows=6, cols=64, groups=2)
    for kw, status in ((dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=16385), 2), (dict(groups=0), 2),
                       (dict(groups=4), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2)):
        p = la.NormProblem(**{**dict(rows=6, cols=64, groups=2), **kw})
        assert fwd(p) == status, kw
        assert la.layernorm_workspace_bytes(p, 148) == 0
    assert fwd(ok, sx=63) == 2 and fwd(ok, sy=0) == 2 and fwd(ok, dtype=5) == 5 and fwd(ok, flags=1) == 5
    assert fwd(ok, x=None) == 1 and fwd(ok, mean=16) == 1
    assert fwd(ok, x=17) == 4 and fwd(ok, w=20) == 4 and fwd(ok, y=(1 << 20) + 1) == 4
    assert fwd(ok, y=32) == 2                       # a shifted overlap
    c = ok.c()
    back = lib.la_layernorm_backward
    assert back(ctypes.byref(c), 16, 16, None, None, 16, 1 << 20, None, None, 16, 0, None) == 1
    assert back(ctypes.byref(c), 16, 16, None, 16, 16, 48, None, None, 16, 0, None) == 2
    c.sdx = 32
    assert back(ctypes.byref(c), 16, 16, None, 16, 16, 1 << 20, None, None, 16, 0, None) == 2


def test_clip_rejects_bad_arguments_before_cuda():
    lib = blk._lib()

    def clip(rows, max_norm=1.0, norm=16, count=None):
        arr = (blk.LaGrad * max(len(rows), 1))(*[blk.LaGrad(*r) for r in rows])
        return lib.la_clip_grad_norm(arr, len(rows) if count is None else count, max_norm, norm, 16, 0, None)

    good = (4096, 4096, 8, 1, 0)
    assert clip([good], norm=None) == 1 and clip([good], norm=18) == 4 and clip([good], count=-1) == 2
    assert clip([good], max_norm=float("nan")) == 2 and clip([good], max_norm=float("inf")) == 2
    assert clip([good], max_norm=-1.0) == 2
    for row, status in (((4096, 4096, 8, 2, 0), 5), ((4096, 4096, 8, 1, 1), 5), ((4096, 4096, -1, 1, 0), 2),
                        ((None, 4096, 8, 1, 0), 1), ((4096, None, 8, 1, 0), 1), ((4098, 4096, 8, 1, 0), 4),
                        ((4096, 4097, 8, 0, 0), 4), ((4096, 4096, BIG * 8, 1, 0), 2)):
        assert clip([row]) == status, row
    assert clip([good, good]) == 2                                            # the same gradient twice, in place
    assert clip([good, (4112, 4112, 8, 1, 0)]) == 2                            # overlapping outputs
    assert clip([(4096, 8192, 8, 1, 0), (8208, 12288, 8, 1, 0)]) == 2          # an output over another input
    assert clip([(4096, 4100, 8, 1, 0)]) == 2                                  # a shifted copy
    assert lib.la_clip_grad_norm(None, 1, 1.0, 16, 16, 0, None) == 1
    assert lib.la_clip_workspace_bytes_for(-1, 148) == 0
    assert lib.la_clip_workspace_bytes_for(2000, 148) > lib.la_clip_workspace_bytes_for(2, 148) > 0


def test_workspaces_grow_with_the_work_and_stay_bounded():
    small = la.cross_workspace_bytes(la.CrossProblem(B=1, H=1, Nq=1, Nk=1), 148)
    split = la.cross_workspace_bytes(la.CrossProblem(B=1, H=8, Nq=1, Nk=16384), 148)
    train = la.cross_workspace_bytes(la.CrossProblem(B=1, H=32, Nq=75600, Nk=300), 148)
    assert 0 < small < split < 1 << 30 and small < train < 1 << 30
    assert la.layernorm_workspace_bytes(la.NormProblem(rows=75600, cols=4096), 148) < 1 << 26


def test_binding_checks_shapes_types_and_devices():
    p = la.CrossProblem(B=1, H=2, Nq=3, Nk=4, d=32)
    Q = torch.zeros((1, 2, 3, 32), dtype=torch.bfloat16)
    K = torch.zeros((1, 2, 4, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        la.cross_forward(p, Q, K, K)
    n = la.NormProblem(rows=3, cols=32)
    with pytest.raises(ValueError, match="CUDA device"):
        la.layernorm_forward(n, Q[0, 0])
    with pytest.raises(ValueError, match="CUDA device"):
        la.grad_norm([Q])
    with pytest.raises(ValueError, match="expected torch.bfloat16 or torch.float32"):
        la.clip_grad_norm([Q.half()], 1.0)
    with pytest.raises(ValueError, match="tensors for"):
        la.clip_grad_norm([Q], 1.0, out=[])


def _differences(f, x, g, seed):
    """Directional derivative of sum(f(x) * g) along a random direction, by central differences."""
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    h = 1e-5
    return float(((f(x + h * d) - f(x - h * d)) * g).sum() / (2 * h)), d


def test_oracle_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, H, Hkv, Nq, Nk, d = 2, 4, 2, 5, 7, 8
    x = [rnd(B, H, Nq, d), rnd(B, Hkv, Nk, d), rnd(B, Hkv, Nk, d)]
    g = rnd(B, H, Nq, d)
    ok = bo.attended(B, Nk, torch.tensor([4, 7]), rnd(B, Nk) > -0.5)
    bo.HALF_STEP[torch.float64] = 0.0
    try:
        grads, _ = bo.cross_backward(*x, g, 0.3, ok)
        for i in range(3):
            f = lambda t: bo.cross_forward(*x[:i], t, *x[i + 1:], 0.3, ok)[0]  # noqa: E731
            num, dirn = _differences(f, x[i], g, i)
            assert abs(num - float((grads[i] * dirn).sum())) < 1e-6 * (1 + abs(num))
        a, w, b, dy = rnd(6, 9), rnd(2, 9), rnd(2, 9), rnd(6, 9)
        (_, mean, rstd), _ = bo.norm_forward(a, w, b, 1e-3)
        grads, _ = bo.norm_backward(a, dy, w, mean, rstd, 2)
        for i, (t, f) in enumerate(((a, lambda t: bo.norm_forward(t, w, b, 1e-3)[0][0]),
                                    (w, lambda t: bo.norm_forward(a, t, b, 1e-3)[0][0]),
                                    (b, lambda t: bo.norm_forward(a, w, t, 1e-3)[0][0]))):
            num, dirn = _differences(f, t, dy, 10 + i)
            assert abs(num - float((grads[i] * dirn).sum())) < 1e-6 * (1 + abs(num))
    finally:
        del bo.HALF_STEP[torch.float64]


def test_oracle_rows_that_see_nothing():
    Q, K = torch.randn(1, 2, 3, 8), torch.full((1, 2, 4, 8), float("nan"))
    ok = bo.attended(1, 4, torch.tensor([0]))
    o, lse, _, _ = bo.cross_forward(Q, K, K, 1.0, ok)
    assert not o.any() and (lse == -float("inf")).all()
    grads, _ = bo.cross_backward(Q, K, K, torch.randn(1, 2, 3, 8), 1.0, ok)
    assert all(not t.any() for t in grads)
