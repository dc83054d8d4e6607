"""Accuracy of head-decay linear attention and of the norm's weight gradients in
relative 2-norm, per tensor and per head (needs a B200; bounds in la_norms)."""
import pytest
import torch

import la_norms
import la_ref
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
