"""Refusals of the operators of the block around the token mixer that need no GPU."""
import ctypes

import pytest

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import block as blk

CROSS = dict(Q=16, K=32, V=48, kv_len=64, key_mask=80, O=96, lse=112)
GRADS = dict(Q=16, K=32, V=48, kv_len=64, key_mask=80, O=96, lse=112, dO=128, dQ=144, dK=160, dV=176)


def _cross(args, p):
    fn = blk._lib().la_cross_backward if "dQ" in args else blk._lib().la_cross_forward
    return fn(ctypes.byref(p.c()), *args.values(), 16, 0, None)


@pytest.mark.parametrize("args,outs", [(CROSS, ("O", "lse")), (GRADS, ("dQ", "dK", "dV"))], ids=("forward", "backward"))
def test_cross_outputs_at_the_address_of_another_tensor(args, outs):
    p = la.CrossProblem(B=2, H=4, Nq=8, Nk=8, d=64)
    for out in outs:
        for other in args:
            if other != out:
                assert _cross({**args, out: args[other]}, p) == 2, (out, other)
    # (different addresses pass this check: what follows needs a device, or finds no workspace)
    assert _cross(args, p) in (6, 7)


def test_cross_tensors_without_elements_have_no_address():
    none = la.CrossProblem(B=2, H=4, Nq=8, Nk=0, d=64)
    assert _cross({**CROSS, "K": 96, "V": 96}, none) in (6, 7)
    assert _cross({**GRADS, "K": 144, "dK": 144, "dV": 144}, none) in (6, 7)


def test_clip_refuses_a_norm_inside_the_gradients():
    lib = blk._lib()

    def clip(rows, norm):
        arr = (blk.LaGrad * len(rows))(*[blk.LaGrad(*r) for r in rows])
        return lib.la_clip_grad_norm(arr, len(rows), 1.0, norm, 16, 0, None)

    inside = (4096, 4096, 8, 1, 0)      # 32 bytes, in place
    moved = (8192, 12288, 8, 1, 0)
    for norm in (4096, 4124, 8192, 8220, 12288, 12316):
        assert clip([moved, inside], norm) == 2, norm
    for norm in (4092, 4128, 8188, 8224, 12284, 12320):
        assert clip([moved, inside], norm) in (6, 7), norm


def test_layernorm_refuses_outputs_over_other_tensors():
    lib = blk._lib()
    p = la.NormProblem(rows=6, cols=64, groups=2)   # weights: 512 bytes, statistics: 24
    c = p.c()
    fwd = dict(x=1 << 20, weight=4096, bias=8192, y=1 << 21, mean=12288, rstd=16384)
    for change in (dict(mean=16384), dict(mean=16400), dict(rstd=12304), dict(mean=4096), dict(rstd=8192 + 496),
                   dict(mean=4096 - 16), dict(y=4096), dict(mean=1 << 20), dict(rstd=1 << 21)):
        assert lib.la_layernorm_forward(ctypes.byref(c), *{**fwd, **change}.values(), None) == 2, change
    bwd = dict(x=1 << 20, dy=1 << 21, weight=4096, mean=12288, rstd=16384, dx=1 << 22, dweight=20480, dbias=24576)
    for change in (dict(dweight=24576), dict(dbias=20480 + 496), dict(dweight=4096), dict(dbias=12304), dict(dweight=16384 - 496),
                   dict(dx=4096), dict(dx=12288), dict(dweight=1 << 20), dict(dbias=1 << 21), dict(dweight=1 << 22)):
        assert lib.la_layernorm_backward(ctypes.byref(c), *{**bwd, **change}.values(), 16, 0, None) == 2, change
    # what is read only may be shared, and neighbours do not overlap: nothing is refused before the device
    # or the workspace is asked for (backward: it has parts, and there is no workspace)
    big = la.NormProblem(rows=4096, cols=64).c()
    bwd = dict(x=1 << 20, dy=1 << 20, weight=4096, mean=1 << 23, rstd=1 << 23, dx=1 << 22, dweight=4096 + 256, dbias=4096 + 512)
    assert lib.la_layernorm_backward(ctypes.byref(big), *bwd.values(), 16, 0, None) in (6, 7)


def test_a_forward_call_does_not_need_the_gradients_workspace():
    size = la.cross_workspace_bytes
    serve = la.CrossProblem(B=8, H=32, Hkv=8, Nq=1, Nk=16384)
    kv = 2 * 8 * 8 * 16384 * 128 * 2
    assert size(serve, 148, backward=False) < 1 << 22          # parts of a few rows; nothing is gathered
    train = la.CrossProblem(B=1, H=32, Nq=75600, Nk=300)
    assert size(train, 148, backward=False, padded=False) == 16  # straight to the output
    assert size(train, 148, backward=False) < 2 * 32 * 304 * 128 * 2 + 4096
    for p in (serve, train, la.CrossProblem(B=2, H=4, Hkv=2, Nq=9, Nk=5000, dtype="f32")):
        whole = size(p, 148)
        assert whole == blk._lib().la_cross_workspace_bytes_for(ctypes.byref(p.c()), 148)
        assert size(p, 148, padded=False) < whole and size(p, 148, backward=False) <= whole
        assert size(p, 148, backward=False, padded=False) <= size(p, 148, backward=False)
    assert size(serve, 148) - size(serve, 148, padded=False) >= kv  # the gathered keys and values
    of = blk._lib().la_cross_workspace_bytes_of
    assert of(ctypes.byref(serve.c()), 16, 148) == 0 and of(ctypes.byref(serve.c()), 1, -1) == 0 and of(None, 1, 148) == 0
