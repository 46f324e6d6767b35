"""The operators of the block around the token mixer where calls are legal but unusual: workspaces on
odd boundaries."""
import pytest
import torch

import gated_linear_attention_relu_b200 as la
from oracle import block_oracle as bo
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
