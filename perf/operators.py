"""Cases of the head-decay linear attention and of the query / key norm with
its rotation: what each operator computes, written in elementary torch
operations (``own`` false) or called through this package (``own`` true).

Head-decay linear attention, one decay per (token, head) or one per head:

    S_t = a_t S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t,      a_t in [-1, 1]

as a chunked forward over fixed-length or packed batches, its backward, and a
single-token step in place on the state.  Norm and rotation, for every head of
the queries and of the keys:

    y = x (c |x|^2 + eps)^(-1/2) * w    (c = 1 for "l2", 1 / d for "rms")

followed by a turn of the first ``rot`` channels' pairs by position * inv_freq.
"""
import random

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 128


# ---- cases -----------------------------------------------------------------


def listed():
    return [
        # one layer's prefill of a training-length batch
        _la("la_fwd", "prefill", 4, 4096, 16, 128, 128),
        # one long document: few (sequence, head) pairs, a long token axis, a state to start from
        _la("la_fwd", "prefill_long", 1, 65536, 32, 128, 128, s0=True),
        # a serving batch of prompts of any length, empty ones among them, one decay per head
        _la("la_fwd", "prefill_packed", 32, 4096, 16, 128, 128, packed=7, alpha="head", s0=True),
        # the smallest call, where latency counts
        _la("la_fwd", "prefill_tiny", 1, 64, 2, 16, 16, dtype="f32", alpha="signed"),
        # one layer's backward of a training step
        _la("la_bwd", "train", 4, 4096, 16, 128, 128),
        # a ragged length in 32 bits, one learned decay per head, gradients through both states
        _la("la_bwd", "train_odd", 2, 1000, 4, 64, 64, dtype="f32", alpha="head", s0=True),
        # one token for each sequence of a large serving batch
        _la("la_step", "step_batch", 256, 1, 32, 128, 128),
        # one token of one sequence
        _la("la_step", "step_single", 1, 1, 16, 128, 128, alpha="head"),
        # queries and keys of a prefill, read in place from the fused projection
        _qk("qk_fwd", "norm_prefill", 16384, 16, 16, 128, 128, "rms", fused=True),
        # queries and shared keys of a few single tokens far into their sequences
        _qk("qk_fwd", "norm_step", 8, 32, 8, 128, 64, "rms", pos=1 << 20, interleaved=True),
        # the backward of a training step
        _qk("qk_bwd", "norm_train", 16384, 16, 16, 128, 128, "rms", fused=True),
        # odd counts in 32 bits, unit-length rows without weights
        _qk("qk_bwd", "norm_train_odd", 777, 6, 2, 64, 64, "l2", dtype="f32", interleaved=True,
            weights=False),
    ]


def _la(op, name, B, T, H, dk, dv, dtype="bf16", alpha="token", packed=0, s0=False):
    # packed: 0, or what the sequences' lengths are drawn from (T is then the longest)
    c = dict(op=op, B=B, T=T, H=H, dk=dk, dv=dv, dtype=dtype, alpha=alpha, packed=packed, s0=s0)
    return dict(c, name=name) if name else c


def _qk(op, name, n, hq, hk, d, rot, norm, dtype="bf16", pos=1 << 15, interleaved=False,
        fused=False, weights=True):
    c = dict(op=op, n=n, hq=hq, hk=hk, d=d, rot=rot, norm=norm, dtype=dtype, pos=pos,
             interleaved=interleaved, fused=fused, weights=weights)
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_bwd", "la_step", "qk_fwd", "qk_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("qk"):
        d = rng.choice([16, 32, 64, 128])
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hq = hk * rng.choice([1, 1, 2, 4])
        n = min(_log(rng, 1, 16384), 16384 * 2048 // (d * hq))
        return _qk(op, None, n, hq, hk, d, rng.choice([0, d // 2, d, d]),
                   rng.choice(["rms", "l2"]), dtype=dtype, pos=_log(rng, 1 << 4, 1 << 20),
                   interleaved=rng.random() < 0.5, fused=rng.random() < 0.5,
                   weights=rng.random() < 0.7)
    alpha = rng.choice(["token", "signed", "head"])
    dk, dv = rng.choice([(128, 128)] * 4 + [(64, 64)] * 2 + [(64, 128), (128, 64), (32, 32),
                                                            (16, 64), (128, 16)])
    if op == "la_step":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        B = min(_log(rng, 1, 256), 8192 // H)
        return _la(op, None, B, 1, H, dk, dv, dtype=dtype, alpha=alpha)
    T = _log(rng, 1, 16384 if op == "la_fwd" else 8192)
    H = rng.choice([1, 2, 3, 4, 8, 16])
    most = (262144 if op == "la_fwd" else 131072) // (1 if dtype == "bf16" else 4)
    B = max(1, min(_log(rng, 1, 48), most // max(1, T * H)))
    packed = rng.randrange(1, 1 << 20) if rng.random() < 0.4 else 0
    return _la(op, None, B, T, H, dk, dv, dtype=dtype, alpha=alpha, packed=packed,
               s0=rng.random() < 0.5)


def _lens(case):
    """The sequences' lengths: one empty, one of a single token, one of T tokens, others between."""
    if not case["packed"]:
        return [case["T"]] * case["B"]
    r = random.Random(case["packed"])
    got = [case["T"], 0, 1][: case["B"]]
    got += [r.randint(0, case["T"]) for _ in range(case["B"] - len(got))]
    r.shuffle(got)
    return got


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("qk"):
        x = case["n"] * (case["hq"] + case["hk"]) * case["d"]
        small = 4 * case["n"] + 2 * case["rot"] + (16 * case["d"] if case["weights"] else 0)
        fwd = case["op"] == "qk_fwd"
        return {"bytes": x * e * (2 if fwd else 3) + small, "flops": x * (8 if fwd else 16)}
    n, H, dk, dv = len(_lens(case)), case["H"], case["dk"], case["dv"]
    th = sum(_lens(case)) * H
    state = n * H * dk * dv * 4
    al = 4 * H if case["alpha"] == "head" else 4 * th
    if case["op"] == "la_fwd":  # q, k, v, decays in; o and the last state out
        return {"bytes": th * (2 * dk + 2 * dv) * e + al + state * (2 if case["s0"] else 1),
                "flops": 4.0 * th * dk * dv}
    if case["op"] == "la_step":  # the state once in and once out
        return {"bytes": th * (2 * dk + 2 * dv) * e + al + 2 * state, "flops": 4.0 * th * dk * dv}
    # q, k, v, do and decays in; dq, dk, dv, the decays' gradient and that of the first state out
    return {"bytes": th * (4 * dk + 3 * dv) * e + 2 * al + state * (3 if case["s0"] else 1),
            "flops": 10.0 * th * dk * dv}


# ---- inputs ----------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if case["op"].startswith("qk"):
        return _prepare_qk(case, g, randn, dt)
    lens = _lens(case)
    B, T, H, dk, dv = len(lens), case["T"], case["H"], case["dk"], case["dv"]
    lead = (sum(lens),) if case["packed"] else (B, T)
    if case["op"] == "la_step":
        lead = (B,)

    def unit(*shape):  # queries and keys come normalised
        x = randn(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = dict(case=case, q=unit(*lead, H, dk), k=unit(*lead, H, dk), v=randn(*lead, H, dv).to(dt))
    # heads forget over 1 to 512 tokens; a signed gate turns the state over now and then, and a
    # zero starts anew
    rate = 2.0 ** -torch.linspace(0, 9, H, device=DEV)
    if case["alpha"] == "head":
        s["alpha"] = torch.exp(-rate * (0.5 + torch.rand(H, generator=g, device=DEV)))
    else:
        a = torch.exp(-rate * torch.nn.functional.softplus(randn(*lead, H)))
        if case["alpha"] == "signed":
            u = torch.rand(a.shape, generator=g, device=DEV)
            a = torch.where(u < 0.25, -a, a)
            a = torch.where(u > 0.995, torch.zeros_like(a), a)
        s["alpha"] = a
    if case["op"] == "la_step":
        s["S"] = 0.3 * randn(B, H, dk, dv)
        return s
    s["S0"] = 0.3 * randn(B, H, dk, dv) if case["s0"] else None
    s["cu"] = None
    if case["packed"]:
        s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    if case["op"] == "la_bwd":
        s["do"] = randn(*lead, H, dv).to(dt)
        s["dSf"] = 0.3 * randn(B, H, dk, dv) if case["s0"] else None
    return s


def _prepare_qk(case, g, randn, dt):
    n, hq, hk, d, rot = (case[x] for x in ("n", "hq", "hk", "d", "rot"))

    def pair():
        if case["fused"]:  # queries, keys and values side by side, as one projection leaves them
            x = randn(n, (hq + 2 * hk) * d).to(dt)
            return x[:, : hq * d].view(n, hq, d), x[:, hq * d: (hq + hk) * d].view(n, hk, d)
        return randn(n, hq, d).to(dt), randn(n, hk, d).to(dt)

    q, k = pair()
    s = dict(case=case, q=q, k=k, wq=None, wk=None, pos=None, freq=None)
    if case["weights"]:
        s["wq"], s["wk"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
    if rot:
        s["pos"] = torch.randint(0, case["pos"], (n,), generator=g, device=DEV, dtype=torch.int32)
        e = torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot
        s["freq"] = (10000.0 ** -e).float()
    if case["op"] == "qk_bwd":
        s["gq"], s["gk"] = randn(n, hq, d).to(dt), randn(n, hk, d).to(dt)
    return s


_EPS = 1e-6


# ---- one pass --------------------------------------------------------------


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import delta_rule_linear_ckda_b200 as ck

        if op == "la_fwd":
            return ck.la_fwd_chunked(s["q"], s["k"], s["v"], s["alpha"], S0=s["S0"],
                                     cu_seqlens=s["cu"])
        if op == "la_step":
            return ck.la_decode_step(s["q"], s["k"], s["v"], s["alpha"], s["S"]), s["S"]
        if op == "la_bwd":
            return ck.la_bwd_chunked(s["q"], s["k"], s["v"], s["alpha"], s["do"], S0=s["S0"],
                                     dS_final=s["dSf"], cu_seqlens=s["cu"])
        if op == "qk_fwd":
            return ck.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], positions=s["pos"],
                                   inv_freq=s["freq"], norm=case["norm"], eps=_EPS,
                                   interleaved=case["interleaved"])
        return ck.qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["wq"], s["wk"],
                                   positions=s["pos"], inv_freq=s["freq"], norm=case["norm"],
                                   eps=_EPS, interleaved=case["interleaved"])
    if op == "la_fwd":
        return _plain_fwd(s)
    if op == "la_bwd":
        return _plain_bwd(s)
    if op == "la_step":
        a = s["alpha"].expand(s["S"].shape[:2])[..., None, None]
        S = a * s["S"] + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
        s["S"].copy_(S)
        return (s["q"].float()[..., :, None] * S).sum(-2).to(s["q"].dtype), s["S"]
    if op == "qk_fwd":
        return (_plain_norm(s, s["q"], s["wq"]).to(s["q"].dtype),
                _plain_norm(s, s["k"], s["wk"]).to(s["q"].dtype))
    dq, dwq = _plain_norm_bwd(s, s["q"], s["gq"], s["wq"])
    dk, dwk = _plain_norm_bwd(s, s["k"], s["gk"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---- the plain forms: linear attention -------------------------------------


def _padded(s):
    """Where each token of a packed batch stands in [N, T]: (index of each padded place, mask)."""
    cu = s["cu"].long()
    at = torch.arange(s["case"]["T"], device=DEV)
    mask = at < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + at).clamp(max=max(0, sum(_lens(s["case"])) - 1)), mask


def _chunks(s, x, places, fill=0.0):
    """[N, H, chunks, C, last] in 32 bits (alpha: 64), places that hold no token filled."""
    x = x if x.dtype == torch.float64 else x.float()
    if places is not None:
        idx, mask = places
        if x.shape[0] == 0:
            x = x.new_zeros((1,) + x.shape[1:])
        x = torch.where(mask[..., None, None], x[idx], torch.full_like(x[:1, :1, :1], fill))
    N, T, H, d = x.shape
    more = -T % _CHUNK
    if more:
        x = torch.cat([x, x.new_full((N, more, H, d), fill)], 1)
    return x.view(N, -1, _CHUNK, H, d).permute(0, 3, 1, 2, 4)


def _unchunk(s, x, places):
    """Back to the input's layout: [N, T, H, last], or [tokens, H, last] of a packed batch."""
    N, H, nc, C, d = x.shape
    x = x.permute(0, 2, 3, 1, 4).reshape(N, nc * C, H, d)[:, : s["case"]["T"]]
    return x[places[1]] if places is not None else x


class _Decay:
    """Products of the decays between positions: logarithms of their sizes, signs and zeros
    summed from the sequence's start in 64 bits."""

    def __init__(self, a):  # [N, H, chunks, C] in 64 bits
        z = a == 0
        flat = a.flatten(2)

        def run_sum(x):
            x = x.double().flatten(2).cumsum(-1)
            return torch.cat([torch.zeros_like(x[..., :1]), x], -1)

        self.parts = (run_sum(torch.where(z, torch.zeros_like(a), torch.where(z, 1, a).abs().log())),
                      run_sum(a < 0), run_sum(z))
        self.T = flat.shape[-1]
        self.nc, self.C = a.shape[2:]

    def at(self, kind):
        """The running sums behind each token ("after"), before it, at the chunks' starts or ends."""
        v = (self.nc, self.C)
        return tuple({"after": p[..., 1:].unflatten(-1, v), "before": p[..., :-1].unflatten(-1, v),
                      "start": p[..., :-1:self.C], "end": p[..., self.C::self.C],
                      "bounds": p[..., ::self.C]}[kind] for p in self.parts)

    @staticmethod
    def between(hi, lo):
        """Product of the decays behind `lo`, up to `hi`; the callers mask lo > hi away."""
        f = torch.exp((hi[0] - lo[0]).clamp(max=0.0))
        f = f * (1 - 2 * torch.remainder(hi[1] - lo[1], 2))
        return torch.where(hi[2] == lo[2], f, torch.zeros_like(f)).float()


def _each(parts, *idx):
    return tuple(p[idx] for p in parts)


def _states(s, dec, k, v, places):
    """The states at the chunks' bounds: [N, H, chunks + 1, dk, dv]."""
    n = (Ellipsis, None)
    w = dec.between(_each(dec.at("end"), *n), dec.at("after"))
    local = (k * w[..., None]).transpose(-1, -2) @ v
    b, e = dec.at("bounds"), dec.at("end")
    m = dec.between(_each(b, ..., slice(None), None), _each(e, ..., None, slice(None)))
    m = m.tril(-1)  # chunk c ends at bound c + 1
    S = (m @ local.flatten(-2)).unflatten(-1, local.shape[-2:])
    if s["S0"] is not None:
        S = S + dec.between(b, _each(b, ..., slice(0, 1)))[..., None, None] * s["S0"][:, :, None]
    return S


def _scores(dec):
    C = _CHUNK
    n = dec.at("after")
    d = dec.between(_each(n, ..., slice(None), None), _each(n, ..., None, slice(None)))
    return d.tril()


def _plain_fwd(s):
    places, (q, k, v, dec) = _inputs(s)
    S = _states(s, dec, k, v, places)
    p = (q @ k.transpose(-1, -2)) * _scores(dec)
    o = p @ v
    pre = dec.between(dec.at("after"), _each(dec.at("start"), ..., None))
    o = o + pre[..., None] * (q @ S[:, :, :-1])
    return _unchunk(s, o, places).to(s["q"].dtype), S[:, :, -1].contiguous()


def _inputs(s):
    places = _padded(s) if s["cu"] is not None else None
    q, k, v = (_chunks(s, s[x], places) for x in "qkv")
    a = s["alpha"].double()
    if a.dim() == 1:
        a = a.expand(s["q"].shape[:-1])
    return places, (q, k, v, _Decay(_chunks(s, a[..., None], places, fill=1.0)[..., 0]))


def _plain_bwd(s):
    places, (q, k, v, dec) = _inputs(s)
    do = _chunks(s, s["do"], places)
    S = _states(s, dec, k, v, places)[:, :, :-1]
    after, before = dec.at("after"), dec.at("before")
    start, end = (_each(dec.at(x), ..., None) for x in ("start", "end"))
    pre, suf = dec.between(after, start)[..., None], dec.between(end, after)[..., None]
    # the states' adjoints at the chunks' bounds
    local = (q * pre).transpose(-1, -2) @ do
    b = dec.at("bounds")
    m = dec.between(_each(dec.at("start"), ..., None, slice(None)), _each(b, ..., slice(None), None))
    G = (m.triu() @ local.flatten(-2)).unflatten(-1, local.shape[-2:])
    if s["dSf"] is not None:
        G = G + dec.between(_each(b, ..., slice(-1, None)), b)[..., None, None] * s["dSf"][:, :, None]
    dS0, G = G[:, :, 0].contiguous(), G[:, :, 1:]
    d = _scores(dec)
    qk, dov = q @ k.transpose(-1, -2), do @ v.transpose(-1, -2)
    sdo, gv, gk = do @ S.transpose(-1, -2), v @ G.transpose(-1, -2), k @ G
    dq = (dov * d) @ k + pre * sdo
    dk = (dov * d).transpose(-1, -2) @ q + suf * gv
    dv = (qk * d).transpose(-1, -2) @ do + suf * gk
    # the decay at t stands in each product over (j, i] with j < t <= i: what is left of it when
    # t is taken out is (t, i] times (j, t - 1]
    one = (Ellipsis, slice(None), None)
    up = dec.between(_each(after, ..., None, slice(None)), _each(after, *one)).triu()
    low = dec.between(_each(before, *one), _each(after, ..., None, slice(None))).tril(-1)
    da = ((up @ (qk * dov)) * low).sum(-1)
    head, tail = dec.between(before, start), dec.between(end, after)
    x, y = (q * sdo).sum(-1), (v * gk).sum(-1)
    da = da + head * (up @ x[..., None])[..., 0] + tail * (low @ y[..., None])[..., 0]
    da = da + head * tail * (S * G).sum((-1, -2))[..., None]
    dt = s["q"].dtype
    dq, dk, dv, da = (_unchunk(s, x, places) for x in (dq, dk, dv, da[..., None]))
    da = da[..., 0].contiguous()
    if s["alpha"].dim() == 1:
        da = da.double().flatten(0, -2).sum(0).float()
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dalpha": da, "dS0": dS0}


# ---- the plain forms: norm and rotation ------------------------------------


def _turned(s, x, back=False):
    """The pairs of the first `rot` channels turned by position * inv_freq (or back)."""
    if s["freq"] is None:
        return x
    rot = 2 * s["freq"].numel()
    ang = s["pos"].double()[:, None, None] * s["freq"].double()
    c, n = ang.cos().float(), ang.sin().float()
    n = -n if back else n
    y = x[..., :rot]
    if s["case"]["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2:]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_norm(s, x, w):
    x = x.float()
    c = 1.0 if s["case"]["norm"] == "l2" else 1.0 / x.shape[-1]
    y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) * c + _EPS)
    return _turned(s, y * w if w is not None else y)


def _plain_norm_bwd(s, x, dy, w):
    dt, x = x.dtype, x.float()
    c = 1.0 if s["case"]["norm"] == "l2" else 1.0 / x.shape[-1]
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) * c + _EPS)
    u = _turned(s, dy.float(), back=True)
    dw = (u * x * r).double().sum((0, 1)).float() if w is not None else None
    u = u * w if w is not None else u
    return (r * u - x * (c * r * r * r) * (x * u).sum(-1, keepdim=True)).to(dt), dw


# ---- the definitions in 64 bits --------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qk"):
        return _exact_qk(s)
    if case["op"] == "la_step":
        S = torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        S += s["S"].double() * s["alpha"].double().expand(s["S"].shape[:2])[:, :, None, None]
        return torch.einsum("bhi,bhij->bhj", s["q"].double(), S), S
    # token by token over sequences side by side; those that have ended stand still
    lens = _lens(case)
    T, B, H = case["T"], len(lens), case["H"]
    first = [sum(lens[:n]) for n in range(B)]

    def lay(x, fill):
        y = torch.full((T, B) + tuple(x.shape[-2:]), float(fill), dtype=torch.float64, device=DEV)
        for n, m in enumerate(lens):
            y[:m, n] = x[first[n]: first[n] + m] if case["packed"] else x[n]
        return y

    def back(y):
        y = [y[:m, n] for n, m in enumerate(lens)]
        return torch.cat(y) if case["packed"] else torch.stack(y)

    a = s["alpha"]
    a = lay((a if a.dim() > 1 else a.expand(s["q"].shape[:-1]))[..., None], 1.0)[..., None]
    q, k, v = (lay(s[x], 0.0) for x in "qkv")
    S = torch.zeros(B, H, case["dk"], case["dv"], dtype=torch.float64, device=DEV)
    if s["S0"] is not None:
        S = s["S0"].double()
    if case["op"] == "la_fwd":
        o = torch.empty_like(v)
        S = S.clone()
        for t in range(T):
            S.mul_(a[t]).addcmul_(k[t][..., :, None], v[t][..., None, :])
            o[t] = (q[t][..., None, :] @ S)[..., 0, :]
        return back(o), S
    do = lay(s["do"], 0.0)
    G = torch.zeros_like(S) if s["dSf"] is None else s["dSf"].double()
    step = 64 if S.numel() <= 1 << 22 else 16
    kept = []
    for t in range(T):
        if t % step == 0:
            kept.append(S)
        S = S * a[t] + k[t][..., :, None] * v[t][..., None, :]
    dq, dk, dv, da = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), \
        torch.empty_like(a)
    for t0 in reversed(range(0, T, step)):
        block = [kept[t0 // step]]
        for t in range(t0, min(T, t0 + step)):
            block.append(block[-1] * a[t] + k[t][..., :, None] * v[t][..., None, :])
        for t in reversed(range(t0, min(T, t0 + step))):
            dq[t] = (block[t - t0 + 1] @ do[t][..., None])[..., 0]
            G = G + q[t][..., :, None] * do[t][..., None, :]
            dk[t] = (G @ v[t][..., None])[..., 0]
            dv[t] = (k[t][..., None, :] @ G)[..., 0, :]
            da[t] = (block[t - t0] * G).sum((-1, -2), keepdim=True)
            G = G * a[t]
    da = back(da[..., 0])[..., 0]
    if s["alpha"].dim() == 1:
        da = da.flatten(0, -2).sum(0)
    return {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dalpha": da, "dS0": G}


def _exact_qk(s):
    """Norm by division and the pairs as complex numbers; the backward through autograd."""
    case = s["case"]
    grads = case["op"] == "qk_bwd"

    def one(x, w, dy):
        d = x.shape[-1]
        x = x.double().requires_grad_(grads)
        w = w.double().requires_grad_(grads) if w is not None else None
        y = x / ((x * x).sum(-1, keepdim=True) / (d if case["norm"] == "rms" else 1) + _EPS).sqrt()
        y = y * w if w is not None else y
        if case["rot"]:
            rot = case["rot"]
            ang = torch.outer(s["pos"].double(), s["freq"].double())[:, None]
            z = y[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
            z = z if case["interleaved"] else z.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(ang), ang))
            z = z if case["interleaved"] else z.transpose(-1, -2)
            y = torch.cat([z.flatten(-2), y[..., rot:]], -1)
        if not grads:
            return y, None
        y.backward(dy.double())
        return x.grad, w.grad if w is not None else None

    q, wq = one(s["q"], s["wq"], s.get("gq"))
    k, wk = one(s["k"], s["wk"], s.get("gk"))
    return {"dq": q, "dk": k, "dwq": wq, "dwk": wk} if grads else (q, k)
