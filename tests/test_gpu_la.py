"""Head-decay linear attention on the GPU against the 64-bit reference of
la_ref (needs a B200): forward, backward and single-token step over types,
head sizes, lengths around every tile's border, packed batches, decays that
are signed, zero, tiny, or one per head, and the ways a caller may run them.
Tolerances are elementwise and derived in la_ref."""
import pytest
import torch

import la_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DIMS = [(16, 16), (32, 64), (64, 32), (128, 16), (64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.fixture(scope="module")
def ck():
    import delta_rule_linear_ckda_b200 as ck

    return ck


def tensor_core(ck, dk, dv, dtype):
    return dtype == torch.bfloat16 and dk in (64, 128) and dv in (64, 128)


def make(lead, H, dk, dv, dtype, decay="token", seed=0, n=None, states=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    q, k, v, dO = r(*lead, H, dk), r(*lead, H, dk), r(*lead, H, dv), r(*lead, H, dv)
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    u = torch.rand((H,) if decay == "head" else (*lead, H), generator=g, device=DEV)
    a = {"token": 0.5 + 0.5 * u, "signed": 2 * u - 1, "head": 0.9 + 0.1 * u, "one": torch.ones_like(u),
         "tiny": 1e-3 * u, "zeros": torch.where(u < 0.1, torch.zeros_like(u), 0.8 + 0.2 * u)}[decay]
    n = lead[0] if n is None else n
    S0, dSf = (0.5 * r(n, H, dk, dv), 0.5 * r(n, H, dk, dv)) if states else (None, None)
    return [x.to(dtype) for x in (q, k, v)] + [a.contiguous(), dO.to(dtype), S0, dSf]


def check_fwd(ck, q, k, v, a, S0, cu=None, out_dtype=None):
    tc = tensor_core(ck, q.shape[-1], v.shape[-1], q.dtype)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu, out_dtype=out_dtype)
    assert ck.device_status() == 0
    ro, rS = la_ref.forward(q, k, v, a, S0, cu)
    to, tS = la_ref.tol_forward(q, k, v, a, o, S0, cu, tensor_core=tc)
    la_ref.check(o, ro, to, "out")
    la_ref.check(S, rS, tS, "S_final")


def check_bwd(ck, q, k, v, a, dO, S0, dSf, cu=None):
    tc = tensor_core(ck, q.shape[-1], v.shape[-1], q.dtype)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    assert ck.device_status() == 0
    ref = la_ref.backward(q, k, v, a, dO, S0, dSf, cu)
    tol = la_ref.tol_backward(q, k, v, a, dO, S0, dSf, cu, tensor_core=tc)
    for n in ref:
        la_ref.check(g[n], ref[n], tol[n], n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_forward_head_sizes(ck, dk, dv, dtype):
    q, k, v, a, _, S0, _ = make((2, 150), 3, dk, dv, dtype, seed=dk + dv)
    check_fwd(ck, q, k, v, a, S0)
    check_fwd(ck, q, k, v, a, None, out_dtype=torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 400])
def test_lengths(ck, T, dtype):
    q, k, v, a, dO, S0, dSf = make((1, T), 2, 128, 128, dtype, "zeros", seed=T)
    check_fwd(ck, q, k, v, a, S0)
    check_bwd(ck, q, k, v, a, dO, S0, dSf)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("decay", ["signed", "head", "one", "tiny", "zeros"])
def test_decays(ck, decay, dtype):
    q, k, v, a, dO, S0, dSf = make((2, 300), 2, 128, 64, dtype, decay, seed=3)
    check_fwd(ck, q, k, v, a, S0)
    check_bwd(ck, q, k, v, a, dO, S0, dSf)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_backward_head_sizes(ck, dk, dv, dtype):
    q, k, v, a, dO, S0, dSf = make((2, 150), 3, dk, dv, dtype, "signed", seed=dk + dv)
    check_bwd(ck, q, k, v, a, dO, S0, dSf)
    check_bwd(ck, q, k, v, a, dO, None, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("decay", ["zeros", "head"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 16)])
def test_packed(ck, dk, dv, decay, dtype):
    lens = [70, 0, 129, 1, 64, 5, 0, 300, 128, 0]
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    q, k, v, a, dO, S0, dSf = make((sum(lens),), 2, dk, dv, dtype, decay, seed=5, n=len(lens))
    check_fwd(ck, q, k, v, a, S0, cu)
    check_bwd(ck, q, k, v, a, dO, S0, dSf, cu)
    _, S = ck.la_fwd_chunked(q[None], k[None], v[None], a if decay == "head" else a[None], S0=S0,
                             cu_seqlens=cu)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    for n, m in enumerate(lens):
        if m == 0:  # nothing runs: the state and its gradient pass through
            assert torch.equal(S[n], S0[n]) and torch.equal(g["dS0"][n], dSf[n])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_that_is_not_finite_leaves_its_neighbours_alone(ck, bad, dtype):
    """A packed batch's tiles reach into the next sequence, a fixed one's into the next row."""
    lens = [100, 37, 200]
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    q, k, v, a, dO, S0, dSf = make((sum(lens),), 2, 128, 128, dtype, seed=6, n=3)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    mid = slice(100, 137)
    for x in (q, k, v, a, dO):
        x[mid] = bad
    o2, S2 = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
    g2 = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    for n, s in ((0, slice(0, 100)), (2, slice(137, 337))):
        assert torch.equal(o[s], o2[s]) and torch.equal(S[n], S2[n])
        for x in ("dq", "dk", "dv", "dalpha"):
            assert torch.equal(g[x][s], g2[x][s]), x
        assert torch.equal(g["dS0"][n], g2["dS0"][n])
    assert not torch.isfinite(S2[1]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_follow_the_forward(ck, dtype):
    """A prompt by the chunked forward, then single tokens, against the whole sequence."""
    q, k, v, a, _, S0, _ = make((3, 140), 2, 128, 128, dtype, "signed", seed=7)
    P = 130
    _, S = ck.la_fwd_chunked(*(x[:, :P].contiguous() for x in (q, k, v, a)), S0=S0)
    outs = [ck.la_decode_step(*(x[:, t].contiguous() for x in (q, k, v, a)), S) for t in range(P, 140)]
    ro, rS = la_ref.forward(q, k, v, a, S0)
    o = torch.stack(outs, 1)
    Mo, MS = la_ref.forward(q, k, v, a, S0, absolute=True)
    m = (2 * 140 + 136) * la_ref.U32
    low = la_ref.UBF if dtype == torch.bfloat16 else 0.0
    tol = m * Mo[:, P:]
    la_ref.check(o, ro[:, P:], tol + low * (ro[:, P:].abs() + 2 * tol), "out")
    la_ref.check(S, rS, m * MS, "S")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (1, 300), (40, 8)])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (128, 32), (64, 64), (128, 128)])
def test_step(ck, dk, dv, B, H, dtype):
    for decay in ("signed", "head"):
        q, k, v, a, _, S0, _ = make((B, 1), H, dk, dv, dtype, decay, seed=B + H, n=B)
        S = S0.clone()
        o = ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                              a if decay == "head" else a[:, 0].contiguous(), S)
        ro, rS = la_ref.forward(q, k, v, a, S0)
        to, tS = la_ref.tol_forward(q, k, v, a, o[:, None], S0)
        la_ref.check(o[:, None], ro, to, "out")
        la_ref.check(S, rS, tS, "S")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_heads_and_long_sequences(ck, dtype):
    """Lengths that a tensor-core call splits into segments; S_final over S0."""
    for B, T, H, dk, dv, lens in ((1, 4500, 2, 128, 128, None), (2, 2200, 1, 64, 64, None),
                                  (3, 5000, 1, 128, 128, [1, 4980, 19])):
        lead, cu = (B, T), None
        if lens:
            lead, cu = (T,), torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        for decay in ("signed", "one"):
            q, k, v, a, _, S0, _ = make(lead, H, dk, dv, dtype, decay, seed=T, n=B)
            check_fwd(ck, q, k, v, a, S0, cu)
            o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
            Sio = S0.clone()
            o2, _ = ck.la_fwd_chunked(q, k, v, a, S0=Sio, S_final=Sio, cu_seqlens=cu)
            assert torch.equal(o, o2) and torch.equal(S, Sio)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (128, 16), (64, 64), (128, 128)])
def test_few_heads_forward_and_backward(ck, dk, dv, dtype):
    """Lengths that a call on the CUDA cores splits into segments, in both directions of time."""
    for lead, lens, decay in (((1, 700), None, "signed"), ((2, 257), None, "zeros"),
                              ((900,), [3, 0, 830, 67], "head"), ((1, 1025), None, "one")):
        cu, n = None, lead[0]
        if lens:
            cu, n = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32), len(lens)
        q, k, v, a, dO, S0, dSf = make(lead, 1, dk, dv, dtype, decay, seed=dk + dv, n=n)
        check_fwd(ck, q, k, v, a, S0, cu)
        check_bwd(ck, q, k, v, a, dO, S0, dSf, cu)
        check_bwd(ck, q, k, v, a, dO, None, None, cu)
        Sio = S0.clone()
        _, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
        ck.la_fwd_chunked(q, k, v, a, S0=Sio, S_final=Sio, cu_seqlens=cu)
        assert torch.equal(S, Sio)


def test_training_sizes_on_sampled_heads(ck):
    B, T, H = 4, 4096, 16
    q, k, v, a, dO, _, _ = make((B, T), H, 128, 128, torch.bfloat16, seed=8, states=False)
    a = torch.exp(-2.0 ** -torch.arange(H, device=DEV).float() * (1 - a)).contiguous()
    o, S = ck.la_fwd_chunked(q, k, v, a)
    g = ck.la_bwd_chunked(q, k, v, a, dO)
    assert ck.device_status() == 0
    for b, h in ((0, 0), (3, 15)):
        sel = lambda x: x[b:b + 1, :, h:h + 1].contiguous()  # noqa: E731
        args = [sel(x) for x in (q, k, v, a)]
        ro, rS = la_ref.forward(*args)
        to, tS = la_ref.tol_forward(*args, sel(o), tensor_core=True)
        la_ref.check(sel(o), ro, to, "out")
        la_ref.check(S[b:b + 1, h:h + 1], rS, tS, "S_final")
        ref = la_ref.backward(*args, sel(dO))
        tol = la_ref.tol_backward(*args, sel(dO), tensor_core=True)
        for n in ("dq", "dk", "dv", "dalpha"):
            la_ref.check(sel(g[n]), ref[n], tol[n], n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_given_whole_deterministic_and_in_place(ck, dtype):
    q, k, v, a, dO, S0, dSf = make((2, 200), 4, 128, 128, dtype, seed=9)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
    out = torch.full_like(v, float("nan"))
    Sio = S0.clone()
    ws = torch.full((max(256, ck.la_workspace_bytes(2, 200, 4, 128, 128, dtype)),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    o2, S2 = ck.la_fwd_chunked(q, k, v, a, S0=Sio, out=out, S_final=Sio, workspace=ws)
    assert o2 is out and S2 is Sio
    assert torch.equal(o, o2) and torch.equal(S, S2)
    pre = {n: torch.full_like(x, float("nan")) for n, x in g.items()}
    ws = torch.full((ck.la_bwd_workspace_bytes(2, 200, 4, 128, 128, False, dtype),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    g2 = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, grads=pre, workspace=ws)
    for n in g:
        assert g2[n] is pre[n] and torch.equal(g[n], g2[n]), n
    g3 = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, want_dS0=False)
    assert g3["dS0"] is None and torch.equal(g["dk"], g3["dk"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_replayed_and_on_another_stream(ck, dtype):
    q, k, v, a, dO, S0, dSf = make((1, 300), 2, 128, 128, dtype, seed=10)
    more = make((1, 300), 2, 128, 128, dtype, seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ck.la_fwd_chunked(q, k, v, a, S0=S0)
        ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
        g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
        St = S.clone()
        y = ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                              a[:, 0].contiguous(), St)
    for src in (more, make((1, 300), 2, 128, 128, dtype, seed=12)):
        for dst, x in zip((q, k, v, a, dO, S0, dSf), src):
            dst.copy_(x)
        graph.replay()
        eo, eS = ck.la_fwd_chunked(q, k, v, a, S0=S0)
        eg = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
        ey = ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                               a[:, 0].contiguous(), eS.clone())
        assert torch.equal(o, eo) and torch.equal(S, eS) and torch.equal(y, ey)
        for n in g:
            assert torch.equal(g[n], eg[n]), n
    assert ck.device_status() == 0


def test_two_calls_at_once(ck):
    cases = [make((2, 700), 4, 128, 128, torch.bfloat16, seed=s) for s in (13, 14)]
    ref = [(ck.la_fwd_chunked(q, k, v, a, S0=S0), ck.la_bwd_chunked(q, k, v, a, dO, S0=S0))
           for q, k, v, a, dO, S0, _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, (q, k, v, a, dO, S0, _) in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append((ck.la_fwd_chunked(q, k, v, a, S0=S0),
                        ck.la_bwd_chunked(q, k, v, a, dO, S0=S0)))
    torch.cuda.synchronize()
    for ((o, S), g), ((ro, rS), rg) in zip(got, ref):
        assert torch.equal(o, ro) and torch.equal(S, rS)
        for n in g:
            assert torch.equal(g[n], rg[n]), n


def test_empty_calls(ck):
    for B, T in ((0, 5), (2, 0), (0, 0)):
        q, k, v, a, dO, S0, dSf = make((B, T), 2, 128, 128, torch.bfloat16)
        o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
        assert o.shape == v.shape and torch.equal(S, S0)
        g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
        assert torch.equal(g["dS0"], dSf)
    a = torch.ones(2, device=DEV)  # one decay per head: its gradient exists without tokens too
    q, k, v, _, dO, S0, dSf = make((2, 0), 2, 32, 32, torch.float32)
    assert torch.equal(ck.la_bwd_chunked(q, k, v, a, dO, S0=S0)["dalpha"], torch.zeros_like(a))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_sequence_leaves_a_zero_gradient_per_head(ck, dtype):
    q, k, v, a, dO, S0, _ = make((0, 5), 2, 128, 128, dtype, "head")
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    for args, c in (((q, k, v, a, dO), None), ((q[:, 0], k[:, 0], v[:, 0], a, dO[:, 0]), cu)):
        g = {"dalpha": torch.full_like(a, float("nan"))}
        ck.la_bwd_chunked(*args, S0=S0, cu_seqlens=c, grads=g)
        assert torch.equal(g["dalpha"], torch.zeros_like(a))


def test_bad_offsets_are_reported(ck):
    q, k, v, a, dO, _, _ = make((200,), 2, 128, 128, torch.bfloat16, states=False)
    for cu in ([0, 120, 90, 200], [0, 100, 180], [5, 100, 200], [0, 300, 200]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        ck.la_fwd_chunked(q, k, v, a, cu_seqlens=cu)
        assert ck.device_status() == -6
        ck.la_bwd_chunked(q, k, v, a, dO, cu_seqlens=cu)
        assert ck.device_status() == -6
    assert ck.device_status() == 0


def test_refusals(ck):
    q, k, v, a, dO, S0, dSf = make((2, 20), 2, 32, 16, torch.bfloat16)
    with pytest.raises(ValueError):
        ck.la_fwd_chunked(q.transpose(1, 2), k, v, a)
    with pytest.raises(ValueError):
        ck.la_fwd_chunked(q, k, v, a[:, :10].contiguous())
    with pytest.raises(TypeError):
        ck.la_fwd_chunked(q, k.float(), v, a)
    with pytest.raises(TypeError):
        ck.la_fwd_chunked(q.half(), k.half(), v.half(), a)
    with pytest.raises(TypeError):
        ck.la_fwd_chunked(q, k, v, a.bfloat16())
    with pytest.raises(ValueError):
        ck.la_fwd_chunked(q, k, v, a, S0=S0[:1].contiguous())
    with pytest.raises(ValueError):
        ck.la_fwd_chunked(q.cpu(), k, v, a)
    with pytest.raises(TypeError):
        ck.la_bwd_chunked(q, k, v, a, dO.float())
    with pytest.raises(ValueError):
        ck.la_bwd_chunked(q, k, v, a, dO, dS_final=S0.transpose(-1, -2).contiguous())
    with pytest.raises(ValueError):
        ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                          a[:1, 0].contiguous(), S0)
    with pytest.raises(ck.CKDAError):
        ck.la_fwd_chunked(q, k, v, a, out=v)
    with pytest.raises(ck.CKDAError):
        ck.la_fwd_chunked(*(x[..., :24].contiguous() for x in (q, k)), v, a)


def test_norm_then_attention_with_gradients(ck):
    """The set as a layer uses it: norm and rotation, attention, single tokens, and back."""
    B, T, H, d = 2, 150, 3, 64
    g = torch.Generator(device=DEV).manual_seed(20)
    x = torch.randn(B, T, 3 * H * d, generator=g, device=DEV)
    xq, xk, v = (x[..., i * H * d:(i + 1) * H * d].view(B, T, H, d) for i in range(3))
    v = v.contiguous()
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    freq = 100.0 ** (-torch.arange(0, d, 2, device=DEV) / d)
    a = 0.9 + 0.1 * torch.rand(B, T, H, generator=g, device=DEV)
    dO = torch.randn(B, T, H, d, generator=g, device=DEV)
    kw = dict(positions=pos, inv_freq=freq, norm="l2")
    q, k = ck.qk_norm_rope(xq, xk, wq, wk, **kw)
    o, S = ck.la_fwd_chunked(q, k, v, a)
    gl = ck.la_bwd_chunked(q, k, v, a, dO)
    gn = ck.qk_norm_rope_bwd(xq, xk, gl["dq"], gl["dk"], wq, wk, **kw)

    # the same in float64 through autograd
    def leaf(t):
        return t.detach().cpu().double().requires_grad_()

    lq, lk, lv, la, lwq, lwk = (leaf(t) for t in (xq, xk, v, a, wq, wk))
    rq, rk = (la_ref.norm_rope(t.reshape(B * T, H, d), w, pos.cpu().reshape(-1), freq.cpu(), "l2")
              .reshape(B, T, H, d) for t, w in ((lq, lwq), (lk, lwk)))
    St, outs = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(T):
        St = la[:, t, :, None, None] * St + rk[:, t, :, :, None] * lv[:, t, :, None, :]
        outs.append((rq[:, t, :, :, None] * St).sum(2))
    ro = torch.stack(outs, 1)
    (ro * dO.cpu().double()).sum().backward()
    # fp32 throughout: a sum's terms pass about 2 T + 4 d roundings; norms of the whole tensors
    bound = (2 * T + 4 * d) * la_ref.U32
    for name, got, ref in (("out", o, ro), ("S", S, St), ("dxq", gn["dq"], lq.grad),
                           ("dxk", gn["dk"], lk.grad), ("dv", gl["dv"], lv.grad),
                           ("dalpha", gl["dalpha"], la.grad), ("dwq", gn["dwq"], lwq.grad),
                           ("dwk", gn["dwk"], lwk.grad)):
        err = (got.cpu().double() - ref).norm() / ref.norm()
        assert err <= bound, (name, float(err))
    # the next token, from the state the forward left
    nq, nk = ck.qk_norm_rope(xq[:, -1], xk[:, -1], wq, wk, positions=pos[:, -1].contiguous(),
                             inv_freq=freq, norm="l2")
    assert torch.equal(nq, q[:, -1]) and torch.equal(nk, k[:, -1])
    _, Sp = ck.la_fwd_chunked(*(t[:, :-1].contiguous() for t in (q, k, v, a)))
    y = ck.la_decode_step(nq, nk, v[:, -1].contiguous(), a[:, -1].contiguous(), Sp)
    assert (y.cpu().double() - ro[:, -1].detach()).norm() <= bound * ro[:, -1].norm()
    # the delta-rule forward takes the same queries and keys
    ck.fwd_chunked(q, k, v, a[..., None].expand(q.shape).contiguous(), a)
    assert ck.device_status() == 0
