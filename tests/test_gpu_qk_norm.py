"""Norm of queries and keys with the rotation on the GPU against the 64-bit
reference of la_ref (needs a B200).  Tolerances: per row, the fp32 steps on an
element's way (a sum of d squares, a square root, three products, the turn)
are below (d + 16) roundings of 2^-24 of the row's largest magnitudes, and a
bf16 result adds one of 2^-8; the angle's rounding is below 2^-22 radians."""
import pytest
import torch

import la_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ck():
    import delta_rule_linear_ckda_b200 as ck

    return ck


def make(n, Hq, Hk, d, rot, dtype, seed=0, fused=False, weights=True, far=1 << 20):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    if fused:
        x = r(n, (Hq + 2 * Hk) * d).to(dtype)
        q, k = x[:, :Hq * d].view(n, Hq, d), x[:, Hq * d:(Hq + Hk) * d].view(n, Hk, d)
    else:
        q, k = r(n, Hq, d).to(dtype), r(n, Hk, d).to(dtype)
    c = dict(wq=None, wk=None, positions=None, inv_freq=None)
    if weights:
        c["wq"], c["wk"] = 1 + 0.2 * r(d), 1 + 0.2 * r(d)
    if rot:
        c["positions"] = torch.randint(-far, far, (n,), generator=g, device=DEV, dtype=torch.int32)
        c["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
                         ).float()
    return q, k, r(n, Hq, d).to(dtype), r(n, Hk, d).to(dtype), c


def ref_fwd(x, w, c, norm, il, eps=1e-6):
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    return la_ref.norm_rope(x, w, cpu(c["positions"]), cpu(c["inv_freq"]), norm, eps, il)


def check(ck, args, norm="rms", il=False, eps=1e-6, out_dtype=None):
    q, k, gq, gk, c = args
    d, dtype = q.shape[-1], q.dtype
    outs = ck.qk_norm_rope(q, k, norm=norm, interleaved=il, eps=eps, out_dtype=out_dtype, **c)
    grads = ck.qk_norm_rope_bwd(q, k, gq, gk, norm=norm, interleaved=il, eps=eps, **c)
    m = (d + 16 + 8) * la_ref.U32
    for x, w, dy, o, dx, dw in ((q, c["wq"], gq, outs[0], grads["dq"], grads["dwq"]),
                                (k, c["wk"], gk, outs[1], grads["dk"], grads["dwk"])):
        assert o.dtype == (out_dtype or dtype) and o.is_contiguous()
        x = x.detach().cpu().double().requires_grad_()
        w = None if w is None else w.detach().cpu().double().requires_grad_()
        y = ref_fwd(x, w, c, norm, il, eps)
        big = y.detach().abs().amax(-1, keepdim=True)  # a pair's turn mixes its two channels
        tol = m * 2 * big + (la_ref.UBF * (y.detach().abs() + m * big)
                             if o.dtype == torch.bfloat16 else 0)
        la_ref.check(o, y.detach(), tol + 1e-30, "out")
        y.backward(dy.cpu().double())
        # dx is a difference of two terms, each below r max|w dy| times a few
        r = y.detach().new_tensor(1.0) / torch.sqrt((x.detach() ** 2).sum(-1, keepdim=True) *
                                                    (1 / d if norm == "rms" else 1.0) + eps)
        wmax = 1.0 if w is None else float(w.detach().abs().max())
        g2 = dy.cpu().double().norm(dim=-1, keepdim=True) * wmax
        size = 2 * r * g2
        tol = m * 2 * size + (la_ref.UBF * x.grad.abs() * 1.01 if dtype == torch.bfloat16 else 0)
        la_ref.check(dx, x.grad, tol + 1e-30, "dx")
        if w is None:
            assert dw is None
        else:
            rows = x.shape[0] * x.shape[1]
            M = (dy.cpu().double().norm(dim=-1, keepdim=True) * (x.detach().abs() * r)).sum((0, 1))
            la_ref.check(dw, w.grad, (d + 24 + rows) * la_ref.U32 * M, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 0), (16, 8), (16, 16), (32, 16), (32, 24), (64, 64), (64, 40),
                                   (128, 128), (128, 64), (128, 8)])
def test_head_sizes_and_turns(ck, d, rot, il, dtype):
    check(ck, make(37, 4, 2, d, rot, dtype, seed=d + rot), il=il)
    check(ck, make(37, 4, 2, d, rot, dtype, seed=d + rot + 1, fused=True, weights=False), "l2", il)


@pytest.mark.parametrize("n,Hq,Hk", [(1, 1, 1), (3, 40, 8), (700, 1, 1), (1000, 3, 1), (5, 2, 0),
                                     (5, 0, 3), (2500, 6, 2)])
def test_counts(ck, n, Hq, Hk):
    check(ck, make(n, Hq, Hk, 64, 32, torch.bfloat16, seed=n))
    check(ck, make(n, Hq, Hk, 128, 128, torch.float32, seed=n, fused=True), "l2")


def test_types_out(ck):
    for dtype in (torch.float32, torch.bfloat16):
        for out in (torch.float32, torch.bfloat16):
            check(ck, make(20, 2, 2, 64, 64, dtype), out_dtype=out)
    q, k, _, _, c = make(20, 2, 2, 64, 64, torch.bfloat16)
    f = ck.qk_norm_rope(q, k, out_dtype=torch.float32, **c)
    b = ck.qk_norm_rope(q, k, **c)
    assert torch.equal(f[0].bfloat16(), b[0]) and torch.equal(f[1].bfloat16(), b[1])


def test_one_weight_only(ck):
    q, k, gq, gk, c = make(50, 3, 2, 32, 16, torch.float32, seed=4)
    c["wk"] = None
    check(ck, (q, k, gq, gk, c))
    c["wq"] = None
    check(ck, (q, k, gq, gk, c))


def test_far_positions(ck):
    """The whole int32 range; a wrong reduction would be off by whole radians."""
    q, k, gq, gk, c = make(64, 2, 1, 32, 32, torch.float32, seed=5)
    c["positions"][:4] = torch.tensor([2**31 - 1, -2**31, 0, 1], device=DEV)
    c["positions"][4:] = torch.randint(-2**31, 2**31 - 1, (60,), device=DEV, dtype=torch.int32)
    check(ck, (q, k, gq, gk, c))


def test_rows_of_zeros_and_tiny_rows(ck):
    q, k, gq, gk, c = make(8, 2, 2, 64, 64, torch.float32, seed=6)
    q[1] = 0
    k[2, 1] = 0
    k[3] *= 1e-12
    check(ck, (q, k, gq, gk, c), "l2")
    o, _ = ck.qk_norm_rope(q, k, norm="l2", eps=0.0, **c)
    g = ck.qk_norm_rope_bwd(q, k, gq, gk, norm="l2", eps=0.0, **c)
    assert torch.equal(o[1], torch.zeros_like(o[1])) and torch.isfinite(g["dwq"]).all()
    assert torch.equal(g["dq"][1], torch.zeros_like(o[1]))


@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_small_rows_without_eps(ck, norm):
    """r = |x|^-1 of these rows is in range, its third power is not."""
    q, k, gq, gk, c = make(12, 2, 2, 64, 64, torch.float32, seed=16)
    check(ck, (q * 1e-15, k * 1e-14, gq, gk, c), norm, eps=0.0)


def test_a_row_that_is_not_finite_stays_alone(ck):
    q, k, gq, gk, c = make(33, 3, 3, 32, 32, torch.bfloat16, seed=7)
    ref = ck.qk_norm_rope(q, k, **c)
    q[5, 1, 3] = float("nan")
    k[6, 0, 0] = float("inf")
    got = ck.qk_norm_rope(q, k, **c)
    keep = torch.ones(33, 3, dtype=torch.bool, device=DEV)
    keep[5, 1] = False
    assert torch.equal(got[0][keep], ref[0][keep]) and torch.isnan(got[0][5, 1]).all()
    keep[5, 1], keep[6, 0] = True, False
    assert torch.equal(got[1][keep], ref[1][keep])


def test_in_place_leading_shapes_and_repeats(ck):
    q, k, gq, gk, c = make(24, 2, 2, 64, 32, torch.bfloat16, seed=8)
    ref = ck.qk_norm_rope(q, k, **c)
    c4 = dict(c, positions=c["positions"].view(4, 6))
    got = ck.qk_norm_rope(q.view(4, 6, 2, 64), k.view(4, 6, 2, 64), **c4)
    assert got[0].shape == (4, 6, 2, 64) and torch.equal(got[0].view_as(q), ref[0])
    g1 = ck.qk_norm_rope_bwd(q, k, gq, gk, **c)
    ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    g2 = ck.qk_norm_rope_bwd(q, k, gq, gk, workspace=ws, **c)
    for n in g1:
        assert torch.equal(g1[n], g2[n])
    a, b = ck.qk_norm_rope(q, k, q_out=q, k_out=k, **c)
    assert a is q and torch.equal(q, ref[0]) and torch.equal(k, ref[1])


def test_captured_and_replayed(ck):
    q, k, gq, gk, c = make(100, 4, 2, 128, 128, torch.bfloat16, seed=9)
    ck.qk_norm_rope(q, k, **c), ck.qk_norm_rope_bwd(q, k, gq, gk, **c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = ck.qk_norm_rope(q, k, **c)
        g = ck.qk_norm_rope_bwd(q, k, gq, gk, **c)
    q.copy_(-2 * q), c["positions"].add_(7)
    graph.replay()
    eo, eg = ck.qk_norm_rope(q, k, **c), ck.qk_norm_rope_bwd(q, k, gq, gk, **c)
    assert torch.equal(o[0], eo[0]) and torch.equal(o[1], eo[1])
    for n in g:
        assert torch.equal(g[n], eg[n])


def test_no_tokens(ck):
    q, k, gq, gk, c = make(0, 2, 2, 32, 16, torch.float32)
    o, _ = ck.qk_norm_rope(q, k, **c)
    assert o.shape == (0, 2, 32)
    g = ck.qk_norm_rope_bwd(q, k, gq, gk, **c)
    assert torch.equal(g["dwq"], torch.zeros(32, device=DEV))


def test_refusals(ck):
    q, k, gq, gk, c = make(6, 2, 2, 32, 16, torch.float32)
    with pytest.raises(ValueError):
        ck.qk_norm_rope(q.transpose(0, 1), k.transpose(0, 1), **dict(c, positions=None, inv_freq=None))
    with pytest.raises(ValueError):
        ck.qk_norm_rope(q, k[:3], **c)
    with pytest.raises(ValueError):
        ck.qk_norm_rope(q, k, **dict(c, inv_freq=None))
    with pytest.raises(TypeError):
        ck.qk_norm_rope(q, k, **dict(c, positions=c["positions"].long()))
    with pytest.raises(TypeError):
        ck.qk_norm_rope(q.half(), k.half(), **c)
    with pytest.raises(ValueError):
        ck.qk_norm_rope(q, k, norm="layer", **c)
    with pytest.raises(ck.CKDAError):
        ck.qk_norm_rope(q, k, eps=-1.0, **c)
    with pytest.raises(ck.CKDAError):
        ck.qk_norm_rope(q, k, **dict(c, inv_freq=c["inv_freq"][:6].contiguous()))  # rot = 12
    with pytest.raises(TypeError):
        ck.qk_norm_rope_bwd(q, k, gq.bfloat16(), gk.bfloat16(), **c)
    with pytest.raises(ck.CKDAError):
        ck.qk_norm_rope(q, k, q_out=k, k_out=q, **c)
