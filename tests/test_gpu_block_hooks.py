"""The hooks build (LA_TEST_HOOKS) of the operators of the block around the token mixer.  The gradients of
cross attention with one of their roles held back: whatever lands or runs late, the results are the
regular library's, bit for bit.  Kernels whose loads never come: their waits run out (here after 65 ms),
they return with the error word set, and the next call is right."""
import ctypes

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import build
from oracle import block_oracle as bo
from test_gpu_block import P_UNIT, close, gen, inputs, rnd

pytestmark = pytest.mark.gpu

HOLD_DO_LOAD, HOLD_DP_ISSUER = 1, 2
LOSE_FORWARD_V, LOSE_DQ_V, LOSE_DKV_DO, LOSE_NORM_ROW = 4, 8, 16, 32
LA_ERR_DEVICE = 8


@pytest.fixture(scope="module")
def hooks(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("hooks") / "liblinattn_hooks.so")
    build.build_variant(out, ["LA_TEST_HOOKS", "LA_WAIT_TESTS=16384u", "LA_WAIT_LIMIT_NS=50000000ull"])
    lib = ctypes.CDLL(out)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.la_cross_forward.argtypes = [vp] * 9 + [sz, vp]
    lib.la_cross_backward.argtypes = [vp] * 13 + [sz, vp]
    lib.la_layernorm_forward.argtypes = [vp] * 8
    lib.la_layernorm_backward.argtypes = [vp] * 10 + [sz, vp]
    lib.la_test_hooks.argtypes = [ctypes.c_uint]
    lib.la_device_error.argtypes = [vp]
    yield lib
    lib.la_test_hooks(0)


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
    assert hooks.la_test_hooks(what) == 0
    try:
        got = [torch.full_like(t, float("nan")) for t in want]
        assert _backward(hooks, p, *args, kv_len, got, ws) == 0
        assert hooks.la_device_error(torch.cuda.current_stream().cuda_stream) == 0
    finally:
        hooks.la_test_hooks(0)
    for a, b, n in zip(got, want, ("dQ", "dK", "dV")):
        assert torch.equal(a, b), n


def _ptrs(*tensors):
    return [None if t is None else t.data_ptr() for t in tensors]


def _cross_calls(d):
    B, H, Hkv, Nq, Nk = 2, 4, 2, 700, 300
    Q, K, V, kv_len, _, ok = inputs(B, H, Hkv, Nq, Nk, d, "bf16", "len")
    dO = rnd((B, H, Nq, d), torch.bfloat16, gen(5))
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d)
    ws = la.cross_workspace(p)
    O, lse = la.cross_forward(p, Q, K, V, kv_len=kv_len, return_lse=True, ws=ws)
    grads = la.cross_backward(p, Q, K, V, O, lse, dO, kv_len=kv_len, ws=ws)

    def forward(lib):
        out = [torch.full_like(O, float("nan")), torch.full_like(lse, float("nan"))]
        c = p.c(**{n: t.stride()[:3] for n, t in zip("qkvo", (Q, K, V, out[0]))})
        rc = lib.la_cross_forward(ctypes.byref(c), *_ptrs(Q, K, V, kv_len, None, *out, ws), ws.numel(),
                                  torch.cuda.current_stream().cuda_stream)
        return rc, out

    def backward(lib):
        out = [torch.full_like(t, float("nan")) for t in grads]
        return _backward(lib, p, Q, K, V, O, lse, dO, kv_len, out, ws), out

    return (forward, (O, lse)), (backward, grads)


def _norm_calls(cols, dtype):
    rows = 4000
    x, dy = (rnd((rows, cols), dtype, gen(i)) for i in (1, 2))
    p = la.NormProblem(rows, cols, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    ws = la.layernorm_workspace(p)
    y, mean, rstd = la.layernorm_forward(p, x, return_stats=True)
    grads = la.layernorm_backward(p, x, dy, mean, rstd, ws=ws)
    c = p.c()

    def forward(lib):
        out = [torch.full_like(t, float("nan")) for t in (y, mean, rstd)]
        return lib.la_layernorm_forward(ctypes.byref(c), *_ptrs(x, None, None, *out), torch.cuda.current_stream().cuda_stream), out

    def backward(lib):
        out = [torch.full_like(t, float("nan")) for t in grads]
        return lib.la_layernorm_backward(ctypes.byref(c), *_ptrs(x, dy, None, mean, rstd, *out, ws), ws.numel(),
                                         torch.cuda.current_stream().cuda_stream), out

    return (forward, (y, mean, rstd)), (backward, grads)


@pytest.mark.parametrize("what,make,which", [
    (LOSE_FORWARD_V, lambda: _cross_calls(128), 0), (LOSE_FORWARD_V, lambda: _cross_calls(64), 0),
    (LOSE_DQ_V, lambda: _cross_calls(128), 1), (LOSE_DQ_V, lambda: _cross_calls(64), 1),
    (LOSE_DKV_DO, lambda: _cross_calls(128), 1), (LOSE_DKV_DO, lambda: _cross_calls(64), 1),
    (LOSE_NORM_ROW, lambda: _norm_calls(8192, torch.bfloat16), 0), (LOSE_NORM_ROW, lambda: _norm_calls(8192, torch.float32), 0),
    (LOSE_NORM_ROW, lambda: _norm_calls(1000, torch.bfloat16), 1), (LOSE_NORM_ROW, lambda: _norm_calls(8192, torch.float32), 1),
], ids=lambda v: str(v) if isinstance(v, int) else "")
def test_a_lost_load_ends_the_kernel_with_an_error(hooks, what, make, which):
    call, want = make()[which]
    stream = torch.cuda.current_stream().cuda_stream
    assert hooks.la_test_hooks(what) == 0
    try:
        rc, _ = call(hooks)
        assert rc == 0 and hooks.la_device_error(stream) == LA_ERR_DEVICE
    finally:
        hooks.la_test_hooks(0)
    rc, got = call(hooks)
    assert rc == 0 and hooks.la_device_error(stream) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert la.device_error() == 0
