"""The 2-norm checks of la_norms reject what they are there for: a gradient of
zeros, one missing term, a scale that is off, and splits into too few bf16
terms; and pass the chunked form with the roundings that the kernels have (CPU).
The mistakes are planted in a chunked form in 64 bits, written out here."""
import pytest
import torch

import la_norms
import la_ref

C, T, H, D = 32, 192, 3, 16


def bf(x):
    return x.bfloat16().double()


def terms(x, n):
    """x as the sum of n bf16 terms (n = 0: unrounded)."""
    if n == 0:
        return x
    s = torch.zeros_like(x)
    for _ in range(n):
        s = s + bf(x - s)
    return s


def case(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k = r(1, T, H, D), r(1, T, H, D)
    q, k = (bf(x / x.norm(dim=-1, keepdim=True)) for x in (q, k))
    a = 0.5 + 0.5 * torch.rand((1, T, H), generator=g, dtype=torch.float64)
    return q, k, bf(r(1, T, H, D)), a, bf(r(1, T, H, D)), 0.5 * r(1, H, D, D), 0.5 * r(1, H, D, D)


def chunked(q, k, v, a, dO, S0, dSf, split=3, score=bf, leave=()):
    """Forward and backward by chunks; ``split``: bf16 terms of the states and of what enters
    them, ``score``: the scores' rounding, ``leave``: terms left out."""
    q, k, v, dO = (x[0].transpose(0, 1) for x in (q, k, v, dO))  # [H, T, D]
    a = a[0].t()
    n = T // C
    ch = lambda x, c: x[:, c * C:(c + 1) * C]  # noqa: E731

    def decays(c):
        x = ch(a, c)
        Dm = torch.zeros(H, C, C, dtype=torch.float64)
        for j in range(C):
            for i in range(j, C):
                Dm[:, i, j] = x[:, j + 1:i + 1].prod(1)
        return Dm, x.cumprod(1), Dm[:, C - 1], x.prod(1)

    Ss, S = [], S0[0]
    for c in range(n):
        _, _, suf, gamma = decays(c)
        Ss.append(S)
        S = gamma[:, None, None] * S + ch(k, c).transpose(1, 2) @ terms(suf[..., None] * ch(v, c), split)
    Gs, G = [None] * n, dSf[0]
    for c in reversed(range(n)):
        _, pre, _, gamma = decays(c)
        Gs[c] = G
        G = gamma[:, None, None] * G + ch(q, c).transpose(1, 2) @ terms(pre[..., None] * ch(dO, c), split)
    r = {"S_final": S[None], "dS0": G[None]}
    cols = {x: [] for x in ("out", "dq", "dk", "dv", "dalpha")}
    for c in range(n):
        Dm, pre, suf, _ = decays(c)
        Q, K, V, O = (ch(x, c) for x in (q, k, v, dO))
        S, G = Ss[c], Gs[c]
        S3, G3 = terms(S, split), terms(G, split)
        s1, s2 = Q @ K.transpose(1, 2), O @ V.transpose(1, 2)
        P, E = score(Dm * s1), score(Dm * s2)
        St, Gt, Et, Pt = S3.transpose(1, 2), score(G).transpose(1, 2), E.transpose(1, 2), P.transpose(1, 2)
        x = (Q * (O @ St)).sum(-1)
        y = (V * (K @ G3)).sum(-1)
        cols["out"].append(P @ V + pre[..., None] * (Q @ score(S)))
        cols["dq"].append(E @ K + pre[..., None] * (O @ St))
        cols["dk"].append(Et @ Q + ("VG" not in leave) * suf[..., None] * (V @ Gt))
        cols["dv"].append(Pt @ O + suf[..., None] * (K @ G3))
        x_, W = ch(a, c), s1 * s2
        da = torch.zeros(H, C, dtype=torch.float64)
        for t in range(C):
            head, tail = x_[:, :t].prod(1), x_[:, t + 1:].prod(1)
            if t > 0:
                da[:, t] += torch.einsum("hi,hj,hij->h", Dm[:, t:, t], Dm[:, t - 1, :t], W[:, t:, :t])
            da[:, t] += head * (Dm[:, t:, t] * x[:, t:]).sum(1)
            if t > 0 and "Y" not in leave:
                da[:, t] += tail * (Dm[:, t - 1, :t] * y[:, :t]).sum(1)
            da[:, t] += ("SG" not in leave) * head * tail * (S * G).sum((1, 2))
        cols["dalpha"].append(da[..., None])
    for name, x in cols.items():
        r[name] = torch.cat(x, 1).transpose(0, 1)[None]
    r["dalpha"] = r["dalpha"][..., 0]
    for name in ("out", "dq", "dk", "dv"):
        r[name] = score(r[name])
    return r


BOUND = {"out": la_norms.LOW, "dq": la_norms.LOW, "dk": la_norms.LOW, "dv": la_norms.LOW,
         "S_final": la_norms.FULL, "dS0": la_norms.FULL, "dalpha": la_norms.FULL}
HEADS = {"out": 2, "dq": 2, "dk": 2, "dv": 2, "S_final": 1, "dS0": 1, "dalpha": 2}


def reference(args):
    q, k, v, a, dO, S0, dSf = args
    r = la_ref.backward(*args)
    r["out"], r["S_final"] = la_ref.forward(q, k, v, a, S0)
    return r


def verdict(got, ref):
    return {n: la_norms.near(got[n], ref[n], b, HEADS[n]) for n, b in BOUND.items()}


def test_the_chunked_form_is_the_recurrence():
    args = case()
    got, ref = chunked(*args, split=0, score=lambda x: x), reference(args)
    for n in BOUND:
        assert la_norms.off(got[n], ref[n]) < 1e-12, n


@pytest.mark.parametrize("seed", [1, 2])
def test_the_kernels_roundings_pass(seed):
    args = case(seed)
    assert all(verdict(chunked(*args), reference(args)).values())


def test_mistakes_are_rejected():
    args = case(3)
    good, ref = chunked(*args), reference(args)
    two = verdict(chunked(*args, split=2), ref)
    assert not two["S_final"] and not two["dS0"] and not two["dalpha"]
    assert not verdict(chunked(*args, split=1), ref)["S_final"]
    assert not verdict(chunked(*args, leave=("Y",)), ref)["dalpha"]
    assert not verdict(chunked(*args, leave=("SG",)), ref)["dalpha"]
    assert not verdict(chunked(*args, leave=("VG",)), ref)["dk"]
    for n in BOUND:
        zero, scaled, one = dict(good), dict(good), dict(good)
        zero[n] = torch.zeros_like(good[n])
        scaled[n] = good[n] * 1.01
        one[n] = good[n].clone()
        one[n].select(HEADS[n], 1).mul_(1.02)
        for x in (zero, scaled, one):
            assert not verdict(x, ref)[n], n
