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
