"""The operators of the block around the token mixer at sizes where a block works on one item after
another, through every kernel that calls choose, on workspaces of odd boundaries and exact sizes, and from
two threads."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import block as blk
from oracle import block_oracle as bo
from test_gpu_block import DT, close, gen, inputs, rnd, unit
from test_gpu_block_use import same_bits

pytestmark = pytest.mark.gpu


# (B, H, Hkv, Nq, Nk, d): whole keys, split keys, a few rows; every kernel with partial sums
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 170, 64), (1, 1, 1, 40, 3000, 128), (2, 4, 2, 1, 5000, 128)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspaces_on_any_16_byte_boundary(shape, dtype):
    """The reported size serves a slice of an arena that starts at 16 of 32 bytes, and no byte around it
    changes; a byte less is refused there."""
    B, H, Hkv, Nq, Nk, d = shape
    Q, K, V, kv_len, mask, _ = inputs(*shape, dtype, "both")
    dO = rnd(Q.shape, DT[dtype], gen(1))
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
    kw = dict(kv_len=kv_len, key_mask=mask)

    def both(ws):
        O, lse = la.cross_forward(p, Q, K, V, return_lse=True, ws=ws, **kw)
        return (O, lse) + la.cross_backward(p, Q, K, V, O, lse, dO, ws=ws, **kw)

    want = both(la.cross_workspace(p))
    n = la.cross_workspace_bytes(p)
    for start in (256, 272, 288, 304):
        arena = torch.full((n + 1024,), 171, dtype=torch.uint8, device="cuda")
        got = both(arena[start:start + n])
        assert all(same_bits(a, b) for a, b in zip(got, want)), start
        assert (arena[:start] == 171).all() and (arena[start + n:] == 171).all()
    with pytest.raises(la.LaError, match="LA_ERR_WORKSPACE"):
        both(arena[272:272 + n - 1])
    with pytest.raises(la.LaError, match="LA_ERR_ALIGN"):
        both(arena[264:264 + n])
    assert la.device_error() == 0


# (the shapes and paths that gather, that read keys where they are, and that split)
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 170, 64), (1, 1, 1, 40, 3000, 128), (2, 4, 2, 1, 5000, 128), (1, 2, 2, 0, 40, 32)],
                         ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", ["none", "len", "mask", "both"])
def test_calls_fit_the_workspace_of_their_own(shape, dtype, pad):
    """Each call stays within the bytes that are reported for it and for what it is given."""
    B, H, Hkv, Nq, Nk, d = shape
    Q, K, V, kv_len, mask, _ = inputs(*shape, dtype, pad)
    dO = rnd(Q.shape, DT[dtype], gen(1))
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
    kw = dict(kv_len=kv_len, key_mask=mask)
    O, lse = la.cross_forward(p, Q, K, V, return_lse=True, ws=la.cross_workspace(p), **kw)
    grads = la.cross_backward(p, Q, K, V, O, lse, dO, ws=la.cross_workspace(p), **kw)
    lib = blk._lib()
    for use, call, want in ((1, lambda ws: la.cross_forward(p, Q, K, V, return_lse=True, ws=ws, **kw), (O, lse)),
                            (2, lambda ws: la.cross_backward(p, Q, K, V, O, lse, dO, ws=ws, **kw), grads)):
        uses = use | (4 if kv_len is not None else 0) | (8 if mask is not None else 0)
        n = lib.la_cross_workspace_bytes_of(ctypes.byref(p.c()), uses, 0)
        assert 16 <= n <= la.cross_workspace_bytes(p)
        arena = torch.full((n + 1024,), 171, dtype=torch.uint8, device="cuda")
        assert all(same_bits(a, b) for a, b in zip(call(arena[272:272 + n]), want))
        assert (arena[:272] == 171).all() and (arena[272 + n:] == 171).all()
        assert all(same_bits(a, b) for a, b in zip(call(None), want))
        if n > 16:
            with pytest.raises(la.LaError, match="LA_ERR_WORKSPACE"):
                call(arena[256:256 + n - 17])
    assert la.device_error() == 0


def test_out_of_memory_is_torchs_error():
    # an output of 8 TB: refused by the allocator, and the next call is right
    huge = la.CrossProblem(B=1, H=1 << 24, Hkv=1 << 24, Nq=1024, Nk=0, d=128)
    one = torch.zeros((1, 1, 1024, 128), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros((1, 1, 0, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        la.cross_forward(huge, one.expand(1, 1 << 24, -1, -1), none.expand(1, 1 << 24, -1, -1), none.expand(1, 1 << 24, -1, -1))
    p = la.CrossProblem(B=1, H=1, Nq=1024, Nk=0, d=128)
    assert not la.cross_forward(p, one, none, none).any()


# (B, H, Hkv, Nq, Nk, d): more work items than SMs in the tensor-core kernels (forward: pairs of query tiles,
# the last of a head with one tile or two; gradients: query tiles, key tiles), shared heads, split keys
ITEMS = [(3, 24, 24, 1100, 300, 128), (3, 24, 8, 1100, 300, 64), (5, 40, 40, 130, 300, 64), (5, 40, 40, 130, 300, 128),
         (3, 32, 32, 513, 260, 32), (1, 100, 50, 200, 2100, 64), (2, 80, 80, 90, 700, 128)]


@pytest.mark.parametrize("pad", ["none", "both", "len"])
@pytest.mark.parametrize("shape", ITEMS, ids=str)
def test_cross_items_one_after_another(shape, pad):
    B, H, Hkv, Nq, Nk, d = shape
    Q, K, V, kv_len, key_mask, ok = inputs(B, H, Hkv, Nq, Nk, d, "bf16", pad, "bnhd" if Nk % 200 else "bhnd")
    dO = rnd((B, H, Nq, d), torch.bfloat16, gen(5), "bnhd")
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d)
    kw = dict(kv_len=kv_len, key_mask=key_mask, ws=la.cross_workspace(p))
    got = la.cross_forward(p, Q, K, V, return_lse=True, **kw)
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok, unit("bf16", False))
    close(got[0], o, to, "O")
    close(got[1], l, tl, "lse")
    args = (Q, K, V, o.to(torch.bfloat16), l.float(), dO)
    grads = la.cross_backward(p, *args, **kw)
    want, tol = bo.cross_backward(Q, K, V, dO, d ** -0.5, ok, unit("bf16", False))
    for a, b, t, n in zip(grads, want, tol, ("dQ", "dK", "dV")):
        close(a, b, t, n)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(la.cross_forward(p, Q, K, V, return_lse=True, **kw), got))
        assert all(torch.equal(a, b) for a, b in zip(la.cross_backward(p, *args, **kw), grads))
    assert la.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", ["mask", "both"])
def test_cross_long_masks_of_several_rows(dtype, pad):
    # masks that are counted in spans first, a length that ends within a span, a row without keys
    B, H, Hkv, Nq, Nk, d = 3, 4, 2, 20, 40001, 64
    Q, K, V, kv_len, key_mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, pad)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
    kw = dict(kv_len=kv_len, key_mask=key_mask)
    O, lse = la.cross_forward(p, Q, K, V, return_lse=True, **kw)
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok, unit(dtype, False))
    close(O, o, to, "O")
    close(lse, l, tl, "lse")
    dO = rnd((B, H, Nq, d), DT[dtype], gen(5))
    got = la.cross_backward(p, Q, K, V, o.to(DT[dtype]), l.float(), dO, **kw)
    want, tol = bo.cross_backward(Q, K, V, dO, d ** -0.5, ok, unit(dtype, False))
    for a, b, t, n in zip(got, want, tol, ("dQ", "dK", "dV")):
        close(a, b, t, n)


# 5 to 8 rows of a key head in one pass
FEW = [(2, 8, 1, 1, 700, 128), (1, 6, 2, 2, 500, 64), (1, 5, 1, 1, 4099, 128), (3, 14, 2, 1, 65, 64), (2, 2, 2, 7, 300, 128)]


@pytest.mark.parametrize("pad", ["none", "both"])
@pytest.mark.parametrize("shape", FEW, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cross_forward_of_five_to_eight_rows(shape, dtype, pad):
    B, H, Hkv, Nq, Nk, d = shape
    Q, K, V, kv_len, key_mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, pad)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
    O, lse = la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=key_mask, return_lse=True)
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok, unit(dtype, False))
    close(O, o, to, "O")
    close(lse, l, tl, "lse")


# (rows, cols, groups): more rows than the few-row kernels take, a width for every kernel of 16-byte packs and
# of single elements; many rows to a block where rows come through a ring
WIDE = [(700, c, 2) for c in (24, 32, 48, 64, 72, 120, 136, 256, 264, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096)] + \
    [(700, c, 1) for c in (7, 31, 127, 301, 1001, 2001, 5001, 10001)] + \
    [(2500, 5000, 1), (2500, 8192, 2), (2400, 16384, 1), (2400, 12296, 3), (6000, 1000, 1), (6000, 4096, 2)]


@pytest.mark.parametrize("shape", WIDE, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_of_many_rows(dtype, shape):
    rows, cols, groups = shape
    g = gen(cols)
    x = (torch.randn((rows, cols), generator=g, device="cuda") * 1.5 + 4.0).to(DT[dtype])
    dy = torch.randn((rows, cols), generator=g, device="cuda").to(DT[dtype])
    w = 1 + 0.2 * torch.randn((groups, cols), generator=g, device="cuda")
    b = torch.randn((groups, cols), generator=g, device="cuda")
    p = la.NormProblem(rows=rows, cols=cols, groups=groups, dtype=dtype)
    got = la.layernorm_forward(p, x, w, b, return_stats=True)
    want, tol = bo.norm_forward(x, w, b, p.eps)
    for a, r, t, n in zip(got, want, tol, ("y", "mean", "rstd")):
        close(a, r, t, n)
    del want, tol
    grads = la.layernorm_backward(p, x, dy, got[1], got[2], w)
    want, tol = bo.norm_backward(x, dy, w, got[1], got[2], groups)
    for a, r, t, n in zip(grads, want, tol, ("dx", "dweight", "dbias")):
        close(a, r, t, n)
    assert all(torch.equal(a, c) for a, c in zip(la.layernorm_forward(p, x, w, b, return_stats=True), got))
    assert all(torch.equal(a, c) for a, c in zip(la.layernorm_backward(p, x, dy, got[1], got[2], w), grads))
    assert la.device_error() == 0


def test_first_call_of_a_host_thread():
    """A thread that has not used CUDA before, and whose call finds everything else in place already."""
    Q, K = (rnd((2, 4, n, 128), torch.bfloat16, gen(n)) for n in (300, 170))
    p = la.CrossProblem(B=2, H=4, Nq=300, Nk=170, d=128)
    ws = la.cross_workspace(p)
    O, lse = la.cross_forward(p, Q, K, K, return_lse=True, ws=ws)
    grads = la.cross_backward(p, Q, K, K, O, lse, Q.clone(), ws=ws)
    dO = Q.clone()
    torch.cuda.synchronize()
    got = []

    def forward():
        got.append(la.cross_forward(p, Q, K, K, return_lse=True, ws=ws, O=torch.empty_like(O)))

    def backward():
        got.append(la.cross_backward(p, Q, K, K, O, lse, dO, ws=ws))

    for call, want in ((forward, (O, lse)), (backward, grads)):
        t = threading.Thread(target=call)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(got) == 1, "the call raised"
        assert all(torch.equal(a, b) for a, b in zip(got.pop(), want))


CAPTURE = """
import torch
import gated_linear_attention_relu_b200 as la
torch.manual_seed(0)
r = lambda *s: torch.randn(s, device="cuda")
Q, K, V, dO = (r(2, 4, n, 64).to(torch.bfloat16) for n in (300, 170, 170, 300))
mask, x, grads = r(2, 170) > 0, r(700, 1000), [r(1000), r(70000).to(torch.bfloat16)]
p, n = la.CrossProblem(B=2, H=4, Nq=300, Nk=170, d=64), la.NormProblem(700, 1000, dtype="f32")
outs = [torch.empty_like(t) for t in grads]

def call():
    O, lse = la.cross_forward(p, Q, K, V, key_mask=mask, return_lse=True)
    y, mean, rstd = la.layernorm_forward(n, x, return_stats=True)
    return (O, lse, *la.cross_backward(p, Q, K, V, O, lse, dO, key_mask=mask), y, mean, rstd,
            *la.layernorm_backward(n, x, x, mean, rstd), la.clip_grad_norm(grads, 1.0, out=outs), *outs)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in captured]
assert all(torch.equal(a, b) for a, b in zip(got, call())) and la.device_error() == 0
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_at_once():
    """Host threads that call into the library at the same time (the C entry points, which take no lock), each
    with a stream and a workspace of its own."""
    lib = blk._lib()
    ptrs = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    jobs = []
    for seed, (B, H, Nq, Nk, d) in enumerate([(2, 6, 300, 170, 64), (1, 4, 700, 1300, 128)]):
        Q, K, V, *_ = inputs(B, H, H, Nq, Nk, d, "bf16", "none", seed=seed)
        dO, x = rnd(Q.shape, torch.bfloat16, gen(seed)), rnd((900, 1000 + 24 * seed), torch.bfloat16, gen(seed))
        p, n = la.CrossProblem(B=B, H=H, Nq=Nq, Nk=Nk, d=d), la.NormProblem(*x.shape)
        O, lse = la.cross_forward(p, Q, K, V, return_lse=True)
        want = [O, lse, *la.cross_backward(p, Q, K, V, O, lse, dO), *la.layernorm_forward(n, x, return_stats=True)]
        want += la.layernorm_backward(n, x, x, want[6], want[7])
        jobs.append((p.c(), n.c(), Q, K, V, O, lse, dO, x, want, [torch.empty_like(t) for t in want],
                     la.cross_workspace(p), la.layernorm_workspace(n), torch.cuda.Stream()))
    torch.cuda.synchronize()
    codes = [[], []]
    start = threading.Barrier(2)

    def work(i):
        c, n, Q, K, V, O, lse, dO, x, want, out, ws, nws, stream = jobs[i]
        st, c, n = stream.cuda_stream, ctypes.byref(c), ctypes.byref(n)
        start.wait()
        for _ in range(100):
            codes[i] += [
                lib.la_cross_forward(c, *ptrs(Q, K, V), None, None, *ptrs(out[0], out[1], ws), ws.numel(), st),
                lib.la_cross_backward(c, *ptrs(Q, K, V), None, None, *ptrs(O, lse, dO, *out[2:5], ws), ws.numel(), st),
                lib.la_layernorm_forward(n, *ptrs(x), None, None, *ptrs(*out[5:8]), st),
                lib.la_layernorm_backward(n, *ptrs(x, x), None, *ptrs(*want[6:8], *out[8:11], nws), nws.numel(), st)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [[0] * 400] * 2
    for job in jobs:
        assert all(torch.equal(a, b) for a, b in zip(job[10], job[9]))
    assert la.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=("f32", "bf16"))
@pytest.mark.parametrize("max_norm", [1e30, 1e9, 1.0, 1e-3, 1e-30])
def test_clipping_by_coefficients_below_fp32s_range(dtype, max_norm):
    """A norm of about 1e40 is beyond fp32 itself, and what clips it may be too; the clipped values are not.
    Half a step of the type, 6 of fp32 for the products and the coefficient, and of the smallest numbers two
    (a product's and the type's)."""
    t = torch.linspace(-3e38, 3e38, 40001, dtype=torch.float64).float().to(dtype).cuda()
    t[:100] = torch.linspace(0.5, 3.0, 100).to(dtype).cuda()
    t[100:200] = torch.linspace(1e-38, 1e-20, 100).to(dtype).cuda()
    ref = float(t.double().square().sum().sqrt())
    want = t.double() * min(1.0, max_norm / (ref + 1e-6))
    smallest = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    for out in (torch.empty_like(t), t):
        la.clip_grad_norm([t], max_norm, out=[out])
        close(out, want, (bo.HALF_STEP[dtype] + 6 * bo.U32) * want.abs() + 2 * smallest, "clipped")
