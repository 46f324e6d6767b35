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
