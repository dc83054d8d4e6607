"""Head-decay linear attention with a single value that is not finite (needs a
B200): it reaches the outputs to which the 64-bit recurrence of la_ref leads
it and no others, whatever lies in the same tile.  An output is compared where
the recurrence leaves it finite; there it does not depend on the value, so the
tolerances are those of the same call without it."""
import pytest
import torch

import la_ref
from test_gpu_la import DEV, ck, make, tensor_core  # noqa: F401

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), float("-inf")]
PLACES = [(3, 5), (40, 15), (127, 0), (128, 9), (200, 2), (299, 11)]  # token, channel


def compare(got, ref, tol, name):
    got, keep = got.detach().cpu().double(), torch.isfinite(ref)
    assert not torch.isfinite(got[~keep]).any(), name
    zero = torch.zeros_like(ref)
    la_ref.check(torch.where(keep, got, zero), torch.where(keep, ref, zero), tol, name)


def spoil(x, t, c, bad):
    """The channel c (or the decay) of token t of the first head."""
    y = x.clone()
    y[(0, t, 0, c) if y.dim() == 4 else (0, t, 0)] = bad
    return y


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 16)])
@pytest.mark.parametrize("which", ["q", "k", "v", "alpha"])
def test_forward(ck, which, dk, dv, dtype):  # noqa: F811
    q, k, v, a, _, S0, _ = make((1, 300), 2, dk, dv, dtype, "signed", seed=dk)
    clean = dict(q=q, k=k, v=v, alpha=a)
    tc = tensor_core(ck, dk, dv, dtype)
    for i, (t, c) in enumerate(PLACES):
        args = dict(clean)
        args[which] = spoil(clean[which], t, c, BAD[i % 3])
        for out_dtype in (dtype, torch.float32):
            o, S = ck.la_fwd_chunked(**args, S0=S0, out_dtype=out_dtype)
            assert ck.device_status() == 0
            to, tS = la_ref.tol_forward(*clean.values(), torch.zeros_like(o), S0, tensor_core=tc)
            ro, rS = la_ref.forward(*args.values(), S0)
            if out_dtype == torch.bfloat16:  # the result's own rounding
                to = to + la_ref.UBF * torch.where(torch.isfinite(ro), ro.abs(), torch.zeros_like(ro))
            compare(o, ro, to, f"out {which} {t}")
            compare(S, rS, tS, f"S_final {which} {t}")


def test_forward_in_segments_and_packed(ck):  # noqa: F811
    """Few heads, so that a sequence runs in segments, and a packed batch's tiles."""
    for lead, lens in (((1, 4500), None), ((1, 700), [100, 37, 363, 200])):
        cu = None if lens is None else \
            torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        n = 1 if lens is None else len(lens)
        q, k, v, a, _, S0, _ = make(lead, 1, 128, 128, torch.bfloat16, "signed", seed=1, n=n)
        to, tS = la_ref.tol_forward(q, k, v, a, v, S0, cu, tensor_core=True)
        for t in (120, 450):
            w = spoil(v, t, 77, float("nan"))
            o, S = ck.la_fwd_chunked(q, k, w, a, S0=S0, cu_seqlens=cu, out_dtype=torch.float32)
            assert ck.device_status() == 0
            ro, rS = la_ref.forward(q, k, w, a, S0, cu)
            compare(o, ro, to, f"out {t}")
            compare(S, rS, tS, f"S_final {t}")


def test_many_values_that_are_not_finite(ck):  # noqa: F811
    """A prompt whose padding holds what memory held: the tokens before it keep their values."""
    q, k, v, a, _, S0, _ = make((3, 400), 2, 128, 64, torch.bfloat16, seed=2)
    ref, _ = ck.la_fwd_chunked(q, k, v, a, S0=S0)
    for b, n in enumerate((1, 130, 333)):
        for x in (q, k, v):
            x[b, n:] = float("nan")
    v[1, 131:] = float("inf")
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
    assert ck.device_status() == 0
    for b, n in enumerate((1, 130, 333)):
        assert torch.equal(o[b, :n], ref[b, :n]) and not torch.isfinite(o[b, n:]).any()
        assert not torch.isfinite(S[b]).any()


def backward_cases(ck, which, dk, dv, dtype):  # noqa: F811
    """(call, 64-bit gradients, tolerances) with one value of ``which`` not finite."""
    q, k, v, a, dO, S0, dSf = make((1, 300), 2, dk, dv, dtype, "signed", seed=dk)
    clean = dict(q=q, k=k, v=v, alpha=a, dO=dO)
    tol = la_ref.tol_backward(*clean.values(), S0, dSf, tensor_core=tensor_core(ck, dk, dv, dtype))
    for i, (t, c) in enumerate(PLACES):
        args = dict(clean)
        args[which] = spoil(clean[which], t, c, BAD[i % 3])
        g = ck.la_bwd_chunked(**args, S0=S0, dS_final=dSf)
        assert ck.device_status() == 0
        yield t, g, la_ref.backward(*args.values(), S0, dSf), tol


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128), (32, 16)])
@pytest.mark.parametrize("which", ["q", "k", "v", "alpha", "dO"])
def test_decays_gradient(ck, which, dk, dv, dtype):  # noqa: F811
    for t, g, ref, tol in backward_cases(ck, which, dk, dv, dtype):
        for n in ("dalpha", "dS0"):
            compare(g[n], ref[n], tol[n], f"{n} {which} {t}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128), (32, 16)])
@pytest.mark.parametrize("which", ["q", "k", "v", "alpha", "dO"])
def test_backward(ck, which, dk, dv, dtype):  # noqa: F811
    for t, g, ref, tol in backward_cases(ck, which, dk, dv, dtype):
        for n in ref:
            compare(g[n], ref[n], tol[n], f"{n} {which} {t}")


def test_backward_after_and_before_other_chunks(ck):  # noqa: F811
    """More (chunk, head) pairs than SMs: the neighbours of a pair with such a value, in the
    same block's walk too, keep their results bit for bit."""
    q, k, v, a, dO, S0, dSf = make((4, 300), 40, 64, 64, torch.bfloat16, "signed", seed=3)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
    w = [x.clone() for x in (q, k, v, dO)]
    hit = torch.zeros(4, 40, dtype=torch.bool, device=DEV)
    for j in range(16):
        b, t, h = j % 4, 37 + 16 * j, (7 * j) % 40
        w[j % 4][b, t, h, j] = BAD[j % 3]
        hit[b, h] = True
    g2 = ck.la_bwd_chunked(w[0], w[1], w[2], a, w[3], S0=S0, dS_final=dSf)
    assert ck.device_status() == 0
    for n in ("dq", "dk", "dv", "dalpha"):
        x, y = (u[n].movedim(1, 2)[~hit] for u in (g, g2))
        assert torch.equal(x, y), n
        assert torch.isfinite(g[n]).all()
    assert torch.equal(g["dS0"][~hit], g2["dS0"][~hit])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_finite_values_pass(ck, dtype):  # noqa: F811
    """Values far above those of other tests, but finite: a power of two scales every result."""
    q, k, v, a, dO, S0, dSf = make((2, 300), 2, 128, 64, dtype, "signed", seed=4)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0)
    f = 2.0 ** 40
    o2, S2 = ck.la_fwd_chunked(q, k, v * f, a, S0=S0 * f)
    g2 = ck.la_bwd_chunked(q, k, v * f, a, dO, S0=S0 * f)
    assert ck.device_status() == 0
    assert torch.equal(o2, o * f) and torch.equal(S2, S * f)
    for n, x in (("dq", f), ("dk", f), ("dv", 1.0), ("dalpha", f), ("dS0", 1.0)):
        assert torch.equal(g2[n], g[n] * x), n
