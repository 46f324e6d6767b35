"""The tensor-core gradients of cross attention with one of their roles held back (the hooks build,
LA_TEST_HOOKS): whatever lands or runs late, the results are the regular library's, bit for bit."""
import ctypes

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import block as blk
from gated_linear_attention_relu_b200 import build
from oracle import block_oracle as bo
from test_gpu_block import P_UNIT, close, gen, inputs, rnd

pytestmark = pytest.mark.gpu

HOLD_DO_LOAD, HOLD_DP_ISSUER = 1, 2


@pytest.fixture(scope="module")
def hooks(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("hooks") / "liblinattn_hooks.so")
    build.build_variant(out, ["LA_TEST_HOOKS"])
    lib = ctypes.CDLL(out)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.la_cross_backward.argtypes = [vp] * 13 + [sz, vp]
    lib.la_test_hold.argtypes = [ctypes.c_uint]
    lib.la_device_error.argtypes = [vp]
    yield lib
    lib.la_test_hold(0)


def _backward(lib, p, Q, K, V, O, lse, dO, kv_len, grads, ws):
    strides = dict(zip(("q", "k", "v", "o", "dout", "dq", "dk", "dv"),
                       (t.stride()[:3] for t in (Q, K, V, O, dO, *grads))))
    c = p.c(**strides)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return lib.la_cross_backward(ctypes.byref(c), *map(ptr, (Q, K, V, kv_len, None, O, lse, dO, *grads, ws)), ws.numel(),
                                 torch.cuda.current_stream().cuda_stream)


# (B, H, Hkv, Nq, Nk, d): one query tile to an item, several, several items to a CTA
@pytest.mark.parametrize("shape", [(1, 2, 2, 100, 300, 128), (2, 2, 1, 700, 200, 128), (2, 12, 6, 520, 1700, 64)], ids=str)
@pytest.mark.parametrize("what", [HOLD_DO_LOAD, HOLD_DP_ISSUER, HOLD_DO_LOAD | HOLD_DP_ISSUER])
def test_a_late_role_changes_nothing(hooks, shape, what):
    B, H, Hkv, Nq, Nk, d = shape
    Q, K, V, kv_len, _, ok = inputs(B, H, Hkv, Nq, Nk, d, "bf16", "len")
    dO = rnd((B, H, Nq, d), torch.bfloat16, gen(5))
    o, l, _, _ = bo.cross_forward(Q, K, V, d ** -0.5, ok)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d)
    ws = la.cross_workspace(p)
    args = (Q, K, V, o.to(torch.bfloat16), l.float(), dO)
    want = la.cross_backward(p, *args, kv_len=kv_len, ws=ws)
    refs, tol = bo.cross_backward(Q, K, V, dO, d ** -0.5, ok, P_UNIT)
    for a, r, t, n in zip(want, refs, tol, ("dQ", "dK", "dV")):
        close(a, r, t, n)
    assert hooks.la_test_hold(what) == 0
    try:
        got = [torch.full_like(t, float("nan")) for t in want]
        assert _backward(hooks, p, *args, kv_len, got, ws) == 0
        assert hooks.la_device_error(torch.cuda.current_stream().cuda_stream) == 0
    finally:
        hooks.la_test_hold(0)
    for a, b, n in zip(got, want, ("dQ", "dK", "dV")):
        assert torch.equal(a, b), n
