"""Plain 64-bit references of head-decay linear attention and of the query /
key norm with its rotation, token by token, and the tolerances that the
kernels' roundings allow (CPU, torch float64).

Tolerances are elementwise.  Each result is a sum of products; with M the same
sum over the terms' absolute values, m roundings on a term's way to the result
move it by at most m u M, u = 2^-24 for fp32 steps and 2^-8 for an operand or
a result rounded to bf16 (first order; the few products of errors are below
one more u).  M is the same recurrence on absolute values.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def _d(x):
    return None if x is None else x.detach().cpu().double()


def spans(q, cu):
    """[(sequence's token index)] over a [tokens, H, d] view."""
    if cu is None:
        B, T = q.shape[:2]
        return [range(b * T, (b + 1) * T) for b in range(B)]
    cu = [int(x) for x in cu.cpu()]
    return [range(a, b) for a, b in zip(cu[:-1], cu[1:])]


def _flat(x, keep):
    return x.reshape((-1,) + tuple(x.shape[-keep:]))


def forward(q, k, v, alpha, S0=None, cu=None, absolute=False):
    """(out shaped like v, S_final [N, H, dk, dv]) in float64."""
    q, k, v, alpha, S0 = (_d(x) for x in (q, k, v, alpha, S0))
    if absolute:
        q, k, v, alpha = q.abs(), k.abs(), v.abs(), alpha.abs()
        S0 = None if S0 is None else S0.abs()
    seqs = spans(q, cu)
    shape = v.shape
    if alpha.dim() == 1:
        alpha = alpha.expand(q.shape[:-1])
    q, k, v, alpha = _flat(q, 2), _flat(k, 2), _flat(v, 2), _flat(alpha, 1)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    out = torch.zeros_like(v)
    last = torch.zeros(len(seqs), H, dk, dv, dtype=torch.float64)
    for n, seq in enumerate(seqs):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[n].clone()
        for t in seq:
            S = alpha[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            out[t] = (q[t][:, :, None] * S).sum(1)
        last[n] = S
    return out.reshape(shape), last


def backward(q, k, v, alpha, dO, S0=None, dSf=None, cu=None, absolute=False):
    """Gradients in float64: dq, dk, dv, dalpha (alpha's shape), dS0."""
    q, k, v, alpha, dO, S0, dSf = (_d(x) for x in (q, k, v, alpha, dO, S0, dSf))
    if absolute:
        q, k, v, alpha, dO = (x.abs() for x in (q, k, v, alpha, dO))
        S0 = None if S0 is None else S0.abs()
        dSf = None if dSf is None else dSf.abs()
    seqs = spans(q, cu)
    shapes = q.shape, v.shape
    per_head = alpha.dim() == 1
    a = alpha.expand(q.shape[:-1]) if per_head else alpha
    q, k, v, dO, a = _flat(q, 2), _flat(k, 2), _flat(v, 2), _flat(dO, 2), _flat(a, 1)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    gq, gk, gv, ga = (torch.zeros_like(x) for x in (q, k, v, a))
    gS = torch.zeros(len(seqs), H, dk, dv, dtype=torch.float64)
    for n, seq in enumerate(seqs):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if S0 is None else S0[n].clone()
        states = [S]
        for t in seq:
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            states.append(S)
        G = torch.zeros_like(S) if dSf is None else dSf[n].clone()
        for i, t in reversed(list(enumerate(seq))):
            gq[t] = (states[i + 1] * dO[t][:, None, :]).sum(2)
            G = G + q[t][:, :, None] * dO[t][:, None, :]
            gk[t] = (G * v[t][:, None, :]).sum(2)
            gv[t] = (G * k[t][:, :, None]).sum(1)
            ga[t] = (G * states[i]).sum((1, 2))
            G = a[t][:, None, None] * G
        gS[n] = G
    ga = ga.sum(0) if per_head else ga.reshape(shapes[0][:-1])
    return {"dq": gq.reshape(shapes[0]), "dk": gk.reshape(shapes[0]), "dv": gv.reshape(shapes[1]),
            "dalpha": ga, "dS0": gS}


def longest(q, cu):
    return max([len(s) for s in spans(q, cu)] + [0])


def tol_forward(q, k, v, alpha, out, S0=None, cu=None, tensor_core=False):
    """(tolerance of out, of S_final): a term passes one rounding per decay and sum
    on its way through the state (2 T), and d_k in the output's sum.  The
    tensor-core form rounds the scores and the state, each once, to bf16."""
    Mo, MS = forward(q, k, v, alpha, S0, cu, absolute=True)
    T, dk = longest(q, cu), q.shape[-1]
    m = (2 * T + dk + 8) * U32
    to = (m + (UBF if tensor_core else 0.0)) * Mo
    if out.dtype == torch.bfloat16:
        to = to + UBF * (out.detach().cpu().double().abs() + to)
    return to + 1e-37, (2 * T + 8) * U32 * MS + 1e-37


def tol_backward(q, k, v, alpha, dO, S0=None, dSf=None, cu=None, tensor_core=False):
    """Per gradient.  dq, dk, dv as the forward's output; dalpha passes both states, the
    sums over d_k and d_v and the chunk's."""
    M = backward(q, k, v, alpha, dO, S0, dSf, cu, absolute=True)
    T, d = longest(q, cu), q.shape[-1] + v.shape[-1]
    m = (2 * T + d + 8) * U32
    low = q.dtype == torch.bfloat16
    t = {n: (m + (UBF if tensor_core else 0.0)) * M[n] for n in ("dq", "dk", "dv")}
    if low:
        t = {n: (1 + UBF) * x + UBF * M[n] for n, x in t.items()}
    t["dalpha"] = (4 * T + 2 * d + 80) * U32 * M["dalpha"]
    if alpha.dim() == 1:
        t["dalpha"] = t["dalpha"] + U32 * M["dalpha"]
    t["dS0"] = (2 * T + 8) * U32 * M["dS0"]
    return {n: x + 1e-37 for n, x in t.items()}


def check(got, ref, tol, name=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{float(got[i])} for {float(ref[i])} (+- {float(tol[i])})")


# ---- norm and rotation -----------------------------------------------------------


def norm_rope(x, w=None, pos=None, freq=None, norm="rms", eps=1e-6, interleaved=False):
    """x [tokens, heads, d] in float64 (kept in the graph)."""
    d = x.shape[-1]
    c = 1.0 / d if norm == "rms" else 1.0
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) * c + eps)
    if w is not None:
        y = y * w
    if freq is None or freq.numel() == 0:
        return y
    rot = 2 * freq.numel()
    ang = pos.double()[:, None, None] * freq.double()
    cs, sn = torch.cos(ang), torch.sin(ang)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = y.clone()
    z[..., a] = y[..., a] * cs - y[..., b] * sn
    z[..., b] = y[..., b] * cs + y[..., a] * sn
    return z
