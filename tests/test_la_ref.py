"""The 64-bit references of la_ref against what fixes them: the oracle's Gated
DeltaNet-2 recurrence with the erase gate off, finite differences, and
closed forms (CPU)."""
import pytest
import torch

import la_ref
import oracle


def _case(B=2, T=7, H=2, dk=5, dv=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    a = torch.rand((B, T, H), generator=g, dtype=torch.float64) * 2 - 1
    return r(B, T, H, dk), r(B, T, H, dk), r(B, T, H, dv), a, r(B, H, dk, dv), r(B, T, H, dv), \
        r(B, H, dk, dv)


def test_forward_is_the_gated_recurrence_without_erasure():
    q, k, v, a, S0, _, _ = _case(dk=16, dv=16)
    q, k, v = (x.float() for x in (q, k, v))
    a, S0 = a.float(), S0.float()
    alpha = a[..., None].expand(q.shape).contiguous()
    o, S = oracle.forward_gdn2(q, k, v, alpha, torch.zeros_like(k), torch.ones_like(v), S0=S0)
    ro, rS = la_ref.forward(q, k, v, a, S0)
    assert torch.allclose(torch.as_tensor(o).reshape(ro.shape), ro, rtol=1e-12, atol=1e-12)
    assert torch.allclose(torch.as_tensor(S).reshape(rS.shape), rS, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("per_head", [False, True])
def test_backward_is_the_forwards_difference_quotient(per_head):
    q, k, v, a, S0, dO, dSf = _case()
    a[0, 3, 0] = 0.0  # a zero decay has its gradient too
    if per_head:
        a = torch.tensor([0.0, -0.7], dtype=torch.float64)
    args = {"dq": q, "dk": k, "dv": v, "dalpha": a, "dS0": S0}
    grads = la_ref.backward(q, k, v, a, dO, S0, dSf)

    def loss():
        o, S = la_ref.forward(q, k, v, a, S0)
        return float((o * dO).sum() + (S * dSf).sum())

    h = 1e-6
    for name, x in args.items():
        flat, g = x.view(-1), grads[name].reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 12)):
            old = float(flat[i])
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            # each value is exact to about 1e-13 of the loss's terms (some hundreds)
            assert abs((up - down) / (2 * h) - float(g[i])) < 1e-5 * max(1.0, abs(float(g[i])))


def test_packed_sequences_start_anew():
    q, k, v, a, _, dO, _ = _case(B=1, T=9)
    cu = torch.tensor([0, 4, 4, 5, 9], dtype=torch.int32)
    o, S = la_ref.forward(q, k, v, a, cu=cu)
    g = la_ref.backward(q, k, v, a, dO, cu=cu)
    assert S.shape[0] == 4 and torch.equal(S[1], torch.zeros_like(S[1]))
    for n, (b, e) in enumerate([(0, 4), (4, 5), (5, 9)]):
        part = [x[:, b:e] for x in (q, k, v, a)]
        assert torch.equal(la_ref.forward(*part)[0], o[:, b:e])
        assert torch.equal(la_ref.backward(*part, dO[:, b:e])["dalpha"], g["dalpha"][:, b:e])


def test_rotation_keeps_lengths_and_depends_on_the_distance_alone():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 2, 16, generator=g, dtype=torch.float64)
    freq = torch.tensor([1.0, 0.3, 0.01, 0.002])
    for il in (False, True):
        rows = [la_ref.norm_rope(x, pos=torch.tensor([p]), freq=freq, interleaved=il)
                for p in (0, 5, 100, 105)]
        for r in rows:
            assert torch.allclose(r.norm(dim=-1), rows[0].norm(dim=-1))
        assert torch.allclose((rows[0] * rows[1]).sum(), (rows[2] * rows[3]).sum())
        assert torch.equal(rows[1][..., 8:], rows[0][..., 8:])
