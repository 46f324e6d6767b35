"""The operators of the block around the token mixer where calls are legal but unusual: workspaces of odd
boundaries and exact sizes, host threads that have not used CUDA."""
import ctypes
import threading

import pytest
import torch

import gated_linear_attention_relu_b200 as la
from gated_linear_attention_relu_b200 import block as blk
from test_gpu_block import DT, gen, inputs, rnd
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
