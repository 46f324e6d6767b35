"""The operators of the block around the token mixer as a program uses them: a whole block with its
gradients and clipping, other streams, captured graphs, views of larger buffers, buffers beyond 2^31
elements, repeated calls."""
import math

import numpy as np
import pytest
import torch

import gated_linear_attention_relu_b200 as la
import oracle as orc
from gated_linear_attention_relu_b200 import workloads as wl
from oracle import block_oracle as bo
from test_gpu_block import DT, P_UNIT, close, gen, inputs, rnd

pytestmark = pytest.mark.gpu


def test_block_forward_backward_and_clipping():
    """A block in fp32: modulated norm -> linear attention -> residual -> norm -> cross attention to a
    padded prompt, its gradients back to the block's input and the norms' parameters, and clipping;
    against the same chain in fp64.  Every operator is within 1e-5 of its largest value (the fp32
    tolerance of the mixer's own tests); four of them in a row, whose norms divide by a standard
    deviation of about 1 and whose softmax and mixer have Lipschitz constants of a few at these sizes,
    stay within 5 * 4 * 1e-5 of the largest."""
    B, H, d, T, Hh, W, Nk = 2, 2, 32, 2, 4, 6, 37
    N, C = T * Hh * W, H * d
    w = wl.custom("block", B=B, H=H, T=T, Hh=Hh, W=W, d=d, bands=(8, 12, 12), dtype="f32")
    p = la.Problem.from_workload(w)
    g = gen(11)
    f = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, K, V, G = f(B * N, C), f(B, H, N, d), f(B, H, N, d), f(B, H, N, d)
    kv = f(B, Nk, 2, H, d)
    Kt, Vt = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    kv_len = torch.tensor([Nk, 5], dtype=torch.int32, device="cuda")
    w1, b1, w2, b2 = 1 + 0.1 * f(B, C), 0.1 * f(B, C), 1 + 0.1 * f(1, C), 0.1 * f(1, C)
    dout = f(B, N, H, d).transpose(1, 2)
    pn1, pn2 = la.NormProblem(B * N, C, groups=B, dtype="f32"), la.NormProblem(B * N, C, dtype="f32")
    pc = la.CrossProblem(B=B, H=H, Nq=N, Nk=Nk, d=d, dtype="f32")
    heads = lambda t: t.view(B, N, H, d).transpose(1, 2)              # noqa: E731
    flat = lambda t: t.transpose(1, 2).reshape(B * N, C)              # noqa: E731

    y1, m1, r1 = la.layernorm_forward(pn1, x, w1, b1, return_stats=True)
    Q = heads(y1).contiguous()
    O1 = la.forward_bidir(p, Q, K, V, G)
    x2 = x + flat(O1)
    y2, m2, r2 = la.layernorm_forward(pn2, x2, w2, b2, return_stats=True)
    out, lse = la.cross_forward(pc, heads(y2), Kt, Vt, kv_len=kv_len, return_lse=True)
    dq, dk, dv = la.cross_backward(pc, heads(y2), Kt, Vt, out, lse, dout, kv_len=kv_len)
    dx2, dw2, db2 = la.layernorm_backward(pn2, x2, flat(dq), m2, r2, w2)
    dQ, dK, dV, dG = la.backward_bidir(p, Q, K, V, G, heads(dx2).contiguous())
    dy1, dw1, db1 = la.layernorm_backward(pn1, x, flat(dQ), m1, r1, w1)
    dx = dx2 + dy1
    grads = [dx, dK, dV, dG, dk.contiguous(), dv.contiguous(), dw1, db1, dw2, db2]
    clipped = [torch.empty_like(t) for t in grads]
    norm = la.clip_grad_norm(grads, 1.0, out=clipped)

    bo.HALF_STEP[torch.float64] = 0.0
    try:
        grid, bands = (T, Hh, W), w.bands
        n64 = lambda t: t.double().cpu().numpy()                      # noqa: E731
        t64 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        ok = bo.attended(B, Nk, kv_len, None, "cuda")
        (ry1, rm1, rr1), _ = bo.norm_forward(x.double(), w1, b1, pn1.eps)
        rO1 = t64(orc.forward_bidir(n64(heads(ry1)), n64(K), n64(V), n64(G), grid, bands, w.rope_base, w.eps))
        rx2 = x.double() + flat(rO1)
        (ry2, rm2, rr2), _ = bo.norm_forward(rx2, w2, b2, pn2.eps)
        rout, rlse, _, _ = bo.cross_forward(heads(ry2), Kt, Vt, d ** -0.5, ok)
        (rdq, rdk, rdv), _ = bo.cross_backward(heads(ry2), Kt.double(), Vt.double(), dout, d ** -0.5, ok)
        (rdx2, rdw2, rdb2), _ = bo.norm_backward(rx2, flat(rdq), w2, rm2, rr2, 1)
        rm = orc.backward_bidir(n64(heads(ry1)), n64(K), n64(V), n64(G), n64(heads(rdx2)), grid, bands, w.rope_base, w.eps)
        rdQ, rdK, rdV, rdG = (t64(a) for a in rm[:4])
        (rdy1, rdw1, rdb1), _ = bo.norm_backward(x.double(), flat(rdQ), w1, rm1, rr1, B)
    finally:
        del bo.HALF_STEP[torch.float64]
    want = [rdx2 + rdy1, rdK, rdV, rdG, rdk, rdv, rdw1, rdb1, rdw2, rdb2]
    for name, a, r in zip(("out", "lse", "dx", "dK", "dV", "dG", "dk", "dv", "dw1", "db1", "dw2", "db2"),
                          [out, lse] + grads, [rout, rlse] + want):
        err = float((a.double() - r).abs().max() / r.abs().max())
        assert err < 2e-4, (name, err)
    total = math.sqrt(sum(float(t.square().sum()) for t in want))
    assert abs(float(norm) - total) < 2e-4 * total
    for a, t in zip(clipped, grads):
        close(a, t.double() * (1.0 / (float(norm) + 1e-6)), 4 * bo.U32 * t.double().abs() + 1e-30, "clipped")
    assert la.device_error() == 0


CALLS = ["cross_tc", "cross_tc_split", "cross_few", "cross_f32", "cross_bwd", "cross_bwd_f32", "norm", "norm_short", "clip"]


def _call(kind, seed):
    """(inputs whose values may change, a call that returns a tuple of outputs) of a kind."""
    if kind.startswith("cross"):
        dtype = "f32" if "f32" in kind else "bf16"
        B, H, Hkv, Nq, Nk, d = {"cross_tc_split": (1, 1, 1, 40, 3000, 128), "cross_few": (2, 4, 2, 1, 5000, 128)}.get(
            kind, (2, 4, 2, 300, 170, 64))
        Q, K, V, kv_len, mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, "both" if Nq > 1 else "len", seed=seed)
        p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
        ws = la.cross_workspace(p)
        if "bwd" not in kind:
            return [Q, K, V], lambda **kw: la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=mask, return_lse=True, ws=ws, **kw)
        dO = rnd(Q.shape, DT[dtype], gen(seed + 1))
        O, lse = la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=mask, return_lse=True)
        return [Q, K, V, O, lse, dO], lambda **kw: la.cross_backward(p, Q, K, V, O, lse, dO, kv_len=kv_len, key_mask=mask,
                                                                     ws=ws, **kw)
    if kind.startswith("norm"):
        rows, cols = (500, 96) if kind == "norm_short" else (400, 4096)
        x, dy = rnd((rows, cols), torch.bfloat16, gen(seed)), rnd((rows, cols), torch.bfloat16, gen(seed + 1))
        w = torch.randn((2, cols), generator=gen(seed + 2), device="cuda")
        p = la.NormProblem(rows, cols, groups=2)
        ws = la.layernorm_workspace(p)

        def both(**kw):
            y, mean, rstd = la.layernorm_forward(p, x, w, return_stats=True, **kw)
            return (y, mean, rstd) + la.layernorm_backward(p, x, dy, mean, rstd, w, ws=ws, **kw)

        return [x, dy, w], both
    grads = [rnd((n,), DT["f32" if i % 2 else "bf16"], gen(seed + i)) for i, n in enumerate((3, 70000, 40001, 8))]
    outs = [torch.empty_like(t) for t in grads]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return grads, lambda **kw: (la.clip_grad_norm(grads, 0.5, out=outs, ws=ws, **kw),) + tuple(outs)


def same_bits(a, b):
    """Equal bit for bit (NaN, where values overflow, included)."""
    kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("kind", CALLS)
def test_other_stream(kind):
    _, call = _call(kind, 1)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):  # the caller's current stream
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", CALLS)
def test_two_captured_graphs(kind):
    # two graphs of the same call, each with its own workspace, replayed in turn on new values
    made = []
    for seed in (1, 2):
        ins, call = _call(kind, seed)
        other, fresh = _call(kind, seed + 20)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        made.append((ins, call, outs, other, graph))
    for k in range(2):
        for ins, call, outs, other, graph in made:
            if k == 1:
                for a, b in zip(ins, other):
                    a.copy_(torch.nan_to_num(b, posinf=0.0, neginf=0.0))
            graph.replay()
        torch.cuda.synchronize()
        for ins, call, outs, other, graph in made:
            got = [t.clone() for t in outs]
            # (what stood in unattended rows may be attended now: some scores overflow)
            assert all(same_bits(a, b) for a, b in zip(got, call()))
    assert la.device_error() == 0


@pytest.mark.parametrize("kind", ["cross_tc", "cross_tc_split", "cross_few", "cross_f32", "cross_bwd", "cross_bwd_f32", "norm"])
def test_many_calls_give_the_same_bits(kind):
    # kernels of a call that start before the ones they depend on have finished would show here
    _, call = _call(kind, 3)
    want = [t.clone() for t in call()]
    for _ in range(60):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_cross_writes_its_rows_only(dtype, d):
    # outputs inside larger buffers, on 16-byte boundaries that are no 32-byte ones
    B, H, Hkv, Nq, Nk = 2, 4, 2, 131, 75
    Q, K, V, kv_len, mask, ok = inputs(B, H, Hkv, Nq, Nk, d, dtype, "both", seed=4)
    p = la.CrossProblem(B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype)
    shift = 16 // Q.element_size()

    def inside(heads, n):
        big = torch.full((B, heads, n + 2, d + 2 * shift), 7.0, dtype=DT[dtype], device="cuda")
        return big, big[:, :, 1:n + 1, shift:shift + d]

    bO, O = inside(H, Nq)
    _, lse = la.cross_forward(p, Q, K, V, kv_len=kv_len, key_mask=mask, O=O, return_lse=True)
    o, l, to, tl = bo.cross_forward(Q, K, V, d ** -0.5, ok, P_UNIT if dtype == "bf16" else 0.0)
    close(O, o, to, "O")
    dO = rnd((B, H, Nq, d), DT[dtype], gen(9))
    bufs = [inside(H, Nq), inside(Hkv, Nk), inside(Hkv, Nk)]
    la.cross_backward(p, Q, K, V, o.to(DT[dtype]), l.float(), dO, kv_len=kv_len, key_mask=mask, grads=[v for _, v in bufs])
    want, tol = bo.cross_backward(Q, K, V, dO, d ** -0.5, ok, P_UNIT if dtype == "bf16" else 0.0)
    for (_, v), r, t, n in zip(bufs, want, tol, ("dQ", "dK", "dV")):
        close(v, r, t, n)
    for big, v in [(bO, O)] + bufs:
        v.fill_(7.0)
        assert (big == 7.0).all()


def test_key_mask_bytes():
    B, H, Nq, Nk, d = 1, 2, 20, 50, 64
    Q, K, V = (rnd((B, H, n, d), torch.bfloat16, gen(n)) for n in (Nq, Nk, Nk))
    p = la.CrossProblem(B=B, H=H, Nq=Nq, Nk=Nk, d=d)
    mask = torch.rand((B, Nk), generator=gen(1), device="cuda") < 0.5
    want = la.cross_forward(p, Q, K, V, key_mask=mask)
    for value in (1, 2, 128, 255):
        assert torch.equal(la.cross_forward(p, Q, K, V, key_mask=mask.to(torch.uint8) * value), want)


@pytest.mark.parametrize("Nq", [1, 24])
def test_cross_offsets_beyond_32_bits(Nq):
    # a cache of more than 2^31 elements per tensor; all but the last keys are left out by the mask (a
    # few rows) or carry little weight (a tile of rows, whose keys are read where they are)
    Nk, d = (1 << 24) + 4099, 128
    K = torch.zeros((1, 1, Nk, d), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    g = gen(6)
    tail = 300
    K[:, :, -tail:] = torch.randn((1, 1, tail, d), generator=g, device="cuda").to(torch.bfloat16)
    V[:, :, -tail:] = torch.randn((1, 1, tail, d), generator=g, device="cuda").to(torch.bfloat16)
    Q = rnd((1, 1, Nq, d), torch.bfloat16, g)
    p = la.CrossProblem(B=1, H=1, Nq=Nq, Nk=Nk, d=d, scale=1.0)
    kw, ok = {}, None
    O, lse = la.cross_forward(p, Q, K, V, return_lse=True, **kw)
    # zero keys: a score of 0 each, a value of 0
    s = (Q.double() @ K[:, :, -tail:].double().transpose(2, 3))
    want = torch.logaddexp(torch.logsumexp(s, 3), torch.tensor(math.log(Nk - tail), device="cuda", dtype=torch.float64))
    o = torch.exp(s - want[..., None]) @ V[:, :, -tail:].double()
    absv = torch.exp(s - want[..., None]) @ V[:, :, -tail:].double().abs()
    # scores up to about 50: 2 (d + 4) 2^-24 |q||k| of them, and a sum of 2^24 terms in parts of at most
    # 2^14 (the splits), each a row of partial sums of 128 or fewer
    per = 2 * (d + 4) * bo.U32 * float((Q.double().abs() @ K[:, :, -tail:].double().abs().transpose(2, 3)).max()) + \
        bo.EXP_U + (2 ** 14 / 128 + 1024 + 128) * bo.U32
    close(lse, want, torch.full_like(want, per + 4 * bo.U32 * float(want.abs().max())), "lse")
    close(O, o, bo.HALF_STEP[torch.bfloat16] * o.abs() + 1.01 * (P_UNIT + per) * absv + 1e-30, "O")
    mask = torch.zeros((1, Nk), dtype=torch.bool, device="cuda")
    mask[:, -tail:] = True
    O = la.cross_forward(p, Q, K, V, key_mask=mask)
    short = la.CrossProblem(B=1, H=1, Nq=Nq, Nk=tail, d=d, scale=1.0)
    o2, _, to, _ = bo.cross_forward(Q, K[:, :, -tail:], V[:, :, -tail:], 1.0,
                                    torch.ones((1, tail), dtype=torch.bool, device="cuda"), P_UNIT)
    close(O, o2, to, "O of the masked cache")
    close(la.cross_forward(short, Q, K[:, :, -tail:], V[:, :, -tail:]), o2, to, "O of its end")


def test_norm_and_clip_beyond_32_bits():
    rows, cols = 530_000, 4096  # 2.2 G elements
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, cols), generator=gen(1), device="cuda").to(torch.bfloat16)
    p = la.NormProblem(rows, cols)
    y, mean, rstd = la.layernorm_forward(p, x, return_stats=True)
    want, tol = bo.norm_forward(x[-3:], None, None, p.eps)
    close(y[-3:], want[0], tol[0], "y")
    dx, dw, db = la.layernorm_backward(p, x, y, mean, rstd)
    want, tol = bo.norm_backward(x[-3:], y[-3:], None, mean[-3:], rstd[-3:], 1)
    close(dx[-3:], want[0], tol[0], "dx")
    close(dw, want[1], tol[1] + 1000 * bo.U32 * want[1].abs(), "dweight")
    x.fill_(0.5)
    flat = x.view(-1)
    n = float(la.clip_grad_norm([flat], 1.0))
    assert abs(n - 0.5 * math.sqrt(rows * cols)) <= 4 * bo.U32 * n
    c = torch.tensor(0.5 / (n + 1e-6)).to(torch.bfloat16)
    assert (flat[-1000:] == c.item()).all() and (flat[:1000] == c.item()).all()


def test_binding_refuses_wrong_tensors():
    p = la.CrossProblem(B=1, H=2, Nq=3, Nk=4, d=32)
    Q, K = torch.zeros((1, 2, 3, 32), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 2, 4, 32), dtype=torch.bfloat16,
                                                                                       device="cuda")
    lse = torch.zeros((1, 2, 3), device="cuda")
    for args, kw, match in (((Q, Q, K), {}, "K: shape"), ((Q.float(), K, K), {}, "Q: torch.Float"),
                            ((Q, K, K), dict(kv_len=torch.zeros(1, device="cuda")), "kv_len"),
                            ((Q, K, K), dict(key_mask=torch.zeros((1, 4), device="cuda")), "key_mask"),
                            ((Q, K, K), dict(key_mask=torch.zeros((1, 8), dtype=torch.bool, device="cuda")[:, ::2]), "contiguous"),
                            ((Q, K, K), dict(lse=lse.double()), "lse"), ((Q, K, K), dict(ws=lse), "ws"),
                            ((Q.transpose(2, 3).contiguous().transpose(2, 3), K, K), {}, "Q: the elements of a row"),
                            ((Q, K, None), {}, "tensors are expected")):
        with pytest.raises(ValueError, match=match):
            la.cross_forward(p, *args, **kw)
    with pytest.raises(la.LaError, match="LA_ERR_WORKSPACE"):
        la.cross_backward(p, Q, K, K, Q.clone(), lse, Q.clone(), ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(la.LaError, match="LA_ERR_ALIGN"):
        big = torch.zeros((1, 2, 3, 36), dtype=torch.bfloat16, device="cuda")
        la.cross_forward(p, big[..., 4:], K, K)
    with pytest.raises(la.LaError, match="LA_ERR_SHAPE"):
        la.cross_forward(p, Q, K, K, O=Q)
    n = la.NormProblem(3, 32)
    x = torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda")
    for kw, match in ((dict(weight=torch.ones(31, device="cuda")), "weight"), (dict(bias=torch.ones(32)), "bias"),
                      (dict(y=x.float()), "y"), (dict(mean=lse), "mean")):
        with pytest.raises(ValueError, match=match):
            la.layernorm_forward(n, x, **kw)
    with pytest.raises(ValueError, match="out 1"):
        la.clip_grad_norm([x, x.clone()], 1.0, out=[x.clone(), x.float()])
    with pytest.raises(ValueError, match="norm"):
        la.grad_norm([x], norm=torch.zeros(2, device="cuda"))
