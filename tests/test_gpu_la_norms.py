"""Accuracy of head-decay linear attention and of the norm's weight gradients in
relative 2-norm, per tensor and per head (needs a B200; bounds in la_norms),
and the walks that only larger calls take: many (chunk, head) pairs per block
of the backward, several units per warp of the norm."""
import pytest
import torch

import la_norms
import la_ref
import test_gpu_qk_norm as qkn
from test_gpu_la import DEV, ck, make, tensor_core  # noqa: F401

pytestmark = pytest.mark.gpu


def check_forward(o, S, ro, rS, tc):
    low = la_norms.LOW if tc else la_norms.ROUND if o.dtype == torch.bfloat16 else la_norms.FULL
    la_norms.check(o, ro, low, "out", -2)
    la_norms.check(S, rS, la_norms.FULL, "S_final", 1)


def check_backward(g, ref, tc):
    for n in ("dq", "dk", "dv"):
        low = la_norms.LOW if tc else \
            la_norms.ROUND if g[n].dtype == torch.bfloat16 else la_norms.FULL
        la_norms.check(g[n], ref[n], low, n, -2)
    la_norms.check(g["dalpha"], ref["dalpha"], la_norms.FULL, "dalpha",
                   -1 if g["dalpha"].dim() > 1 else None)
    if ref.get("dS0") is not None:
        la_norms.check(g["dS0"], ref["dS0"], la_norms.FULL, "dS0", 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [37, 400])
def test_accuracy(ck, T, dk, dv, dtype):  # noqa: F811
    tc = tensor_core(ck, dk, dv, dtype)
    q, k, v, a, dO, S0, dSf = make((2, T), 3, dk, dv, dtype, seed=dk + dv + T)
    for s0, sf in ((S0, dSf), (None, None)):
        check_forward(*ck.la_fwd_chunked(q, k, v, a, S0=s0), *la_ref.forward(q, k, v, a, s0), tc)
        check_backward(ck.la_bwd_chunked(q, k, v, a, dO, S0=s0, dS_final=sf),
                       la_ref.backward(q, k, v, a, dO, s0, sf), tc)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accuracy_of_long_sequences(ck, dtype):  # noqa: F811
    """Decays near one, so that a state holds thousands of tokens."""
    q, k, v, a, dO, _, _ = make((1, 4096), 2, 128, 128, dtype, seed=8, states=False)
    a = torch.exp(-2.0 ** -torch.tensor([3.0, 15.0], device=DEV) * (1 - a)).contiguous()
    tc = dtype == torch.bfloat16
    check_forward(*ck.la_fwd_chunked(q, k, v, a), *la_ref.forward(q, k, v, a), tc)
    ref = la_ref.backward(q, k, v, a, dO)
    ref["dS0"] = None
    check_backward(ck.la_bwd_chunked(q, k, v, a, dO), ref, tc)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_packed_backward_of_many_chunks(ck, dk, dv):  # noqa: F811
    """More (chunk, head) pairs than blocks: whole and partial chunks and empty slots follow one
    another in a block.  Every sequence's gradients equal those of a call on it alone."""
    g = torch.Generator().manual_seed(dk + dv)
    lens = [0, 400, 1] + torch.randint(0, 400, (37,), generator=g).tolist()
    lens[10] = lens[11] = 0
    lens[20], lens[21] = 128, 256
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    H, n = 8, len(lens)
    q, k, v, a, dO, S0, dSf = make((sum(lens),), H, dk, dv, torch.bfloat16, seed=21, n=n)
    got = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    assert ck.device_status() == 0
    bounds = cu.tolist()
    for i in range(n):
        s = slice(bounds[i], bounds[i + 1])
        part = [x[s][None].contiguous() for x in (q, k, v, a, dO)]
        one = ck.la_bwd_chunked(*part, S0=S0[i:i + 1], dS_final=dSf[i:i + 1])
        for x in ("dq", "dk", "dv", "dalpha"):
            assert torch.equal(got[x][s], one[x][0]), (x, i)
        assert torch.equal(got["dS0"][i], one["dS0"][0])
        if i in (1, 2, 5, 20, 39):
            check_backward({x: got[x][s][None] if x != "dS0" else got[x][i:i + 1] for x in got},
                           la_ref.backward(*part, S0[i:i + 1], dSf[i:i + 1]), True)


def test_backward_repeats_itself(ck):  # noqa: F811
    q, k, v, a, dO, _, _ = make((2, 1500), 16, 128, 128, torch.bfloat16, seed=22, states=False)
    o, S = ck.la_fwd_chunked(q, k, v, a)
    g = ck.la_bwd_chunked(q, k, v, a, dO)
    for _ in range(5):
        o2, S2 = ck.la_fwd_chunked(q, k, v, a)
        g2 = ck.la_bwd_chunked(q, k, v, a, dO)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("n,Hq,Hk,d,rot,dtype,il", [
    (6000, 20, 4, 128, 128, torch.bfloat16, False),  # two batches of rows, two units per warp
    (4000, 12, 3, 128, 64, torch.float32, True),
    (3700, 36, 1, 64, 64, torch.bfloat16, False),
    (9001, 5, 5, 16, 8, torch.float32, False),
])
def test_norm_of_many_tokens(ck, n, Hq, Hk, d, rot, dtype, il):  # noqa: F811
    args = qkn.make(n, Hq, Hk, d, rot, dtype, seed=n)
    qkn.check(ck, args, il=il)
    q, k, gq, gk, c = args
    g = ck.qk_norm_rope_bwd(q, k, gq, gk, interleaved=il, **c)
    for x, w, dy, dx, dw in ((q, c["wq"], gq, g["dq"], g["dwq"]),
                             (k, c["wk"], gk, g["dk"], g["dwk"])):
        x, w = (t.detach().cpu().double().requires_grad_() for t in (x, w))
        qkn.ref_fwd(x, w, c, "rms", il).backward(dy.cpu().double())
        la_norms.check(dw, w.grad, la_norms.DW, "dw")
        la_norms.check(dx, x.grad, la_norms.ROUND if dtype == torch.bfloat16 else la_norms.DW, "dx", 1)
    again = ck.qk_norm_rope_bwd(q, k, gq, gk, interleaved=il, **c)
    assert all(torch.equal(g[x], again[x]) for x in g)
