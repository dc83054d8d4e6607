"""Head-decay linear attention and the query / key norm at the ends of what the
documentation allows (needs a B200): many heads, many sequences, tensors of
more than 2^31 elements, packed batches without tokens, a graph whose offsets
change between replays, results of another type than the inputs."""
import pytest
import torch

import la_norms
import la_ref
from test_gpu_la import DEV, ck, make  # noqa: F401
from test_gpu_la_norms import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,T", [(torch.float32, 16, 2), (torch.bfloat16, 64, 3)])
def test_most_heads(ck, dtype, d, T):  # noqa: F811
    H, tc = 65535, dtype == torch.bfloat16
    q, k, v, a, dO, S0, dSf = make((1, T), H, d, d, dtype, seed=1)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf)
    y = ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                          a[:, 0].contiguous(), S1 := S0.clone())
    assert ck.device_status() == 0
    at = torch.tensor([0, 1, 4095, 32768, 65533, 65534], device=DEV)
    q, k, v, a, dO = (x[:, :, at] for x in (q, k, v, a, dO))
    S0, dSf = S0[:, at], dSf[:, at]
    check_forward(o[:, :, at], S[:, at], *la_ref.forward(q, k, v, a, S0), tc)
    check_backward({n: x[:, at] if n == "dS0" else x[:, :, at] for n, x in g.items()},
                   la_ref.backward(q, k, v, a, dO, S0, dSf), tc)
    ro, rS = la_ref.forward(*(x[:, :1] for x in (q, k, v, a)), S0)
    check_forward(y[:, None, at], S1[:, at], ro, rS, False)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 64)])
def test_many_sequences(ck, dtype, d):  # noqa: F811
    """More sequences than are ordered by length, some of them empty."""
    gen = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 9, (1500,), generator=gen).tolist()
    lens[700] = 300
    cu = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    q, k, v, a, dO, S0, dSf = make((sum(lens),), 2, d, d, dtype, seed=2, n=len(lens))
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    assert ck.device_status() == 0
    tc = dtype == torch.bfloat16
    check_forward(o, S, *la_ref.forward(q, k, v, a, S0, cu), tc)
    check_backward(g, la_ref.backward(q, k, v, a, dO, S0, dSf, cu), tc)


def test_offsets_past_31_bits(ck):  # noqa: F811
    """2.2e9 elements per tensor; the first and the last head against calls on them alone, which
    split their sequence into segments."""
    T, H, d = 131077, 130, 128
    gen = torch.Generator(device=DEV).manual_seed(3)

    def rand():
        x = torch.empty((1, T, H, d), dtype=torch.bfloat16, device=DEV)
        return x.normal_(generator=gen).mul_(d ** -0.5)

    q, k, v, dO = (rand() for _ in range(4))
    a = 0.9 + 0.1 * torch.rand((1, T, H), generator=gen, device=DEV)
    assert q.numel() > 2 ** 31
    o, S = ck.la_fwd_chunked(q, k, v, a)
    g = ck.la_bwd_chunked(q, k, v, a, dO)
    assert ck.device_status() == 0
    for h in (0, H - 1):
        part = [x[:, :, h:h + 1].contiguous() for x in (q, k, v, a, dO)]
        o1, S1 = ck.la_fwd_chunked(*part[:4])
        g1 = ck.la_bwd_chunked(*part)
        s = slice(h, h + 1)
        # two results with roundings of their own
        la_norms.check(o[:, :, s], o1, 2 * la_norms.LOW, "out")
        la_norms.check(S[:, s], S1, 2 * la_norms.FULL, "S_final")
        for n in ("dq", "dk", "dv", "dalpha"):
            assert torch.equal(g[n][:, :, s], g1[n]), n
        # the first and the last tokens against the definition, the last ones from a state that
        # holds the tokens before (0.95^500 of what lies further back)
        head = [x[:, :200] for x in part]
        la_norms.check(o[:, :200, s], la_ref.forward(*head[:4])[0], la_norms.LOW, "first")
        tail = [x[:, -900:] for x in part]
        ro, rS = la_ref.forward(*tail[:4])
        la_norms.check(o[:, -300:, s], ro[:, -300:], la_norms.LOW, "last")
        la_norms.check(S[:, s], rS, la_norms.FULL, "S_final")
    del q, k, v, dO, o, g
    torch.cuda.empty_cache()


def test_norm_past_31_bits(ck):  # noqa: F811
    n, H, d = 2 ** 21 + 3, 8, 128
    gen = torch.Generator(device=DEV).manual_seed(4)
    q, gq = (torch.empty((n, H, d), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
             for _ in range(2))
    k, gk = q[:, :1].contiguous(), gq[:, :1].contiguous()
    w = 1 + 0.1 * torch.rand(d, generator=gen, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freq = 10000.0 ** (-torch.arange(0, d, 2, device=DEV) / d)
    o, ok = ck.qk_norm_rope(q, k, w, w, pos, freq)
    g = ck.qk_norm_rope_bwd(q, k, gq, gk, w, w, pos, freq)
    assert torch.equal(o[:, :1], ok) and torch.equal(g["dq"][:, :1], g["dk"])
    for s in (slice(0, 40), slice(n - 40, n)):
        x = q[s].cpu().double().requires_grad_()
        y = la_ref.norm_rope(x, w.cpu().double(), pos[s].cpu(), freq.cpu())
        la_norms.check(o[s], y.detach(), la_norms.ROUND, "out", 1)
        y.backward(gq[s].cpu().double())
        la_norms.check(g["dq"][s], x.grad, la_norms.ROUND, "dq", 1)
    # the weight's gradient of the same rows in 64 bits
    dw = torch.zeros(d, dtype=torch.float64, device=DEV)
    fr = freq.double()
    for b in range(0, n, 1 << 17):
        s = slice(b, min(n, b + (1 << 17)))
        x, y = q[s].double(), gq[s].double()
        ang = pos[s].double()[:, None, None] * fr
        cs, sn = torch.cos(ang), torch.sin(ang)
        y0, y1 = y[..., :d // 2], y[..., d // 2:]
        u = torch.cat([y0 * cs + y1 * sn, y1 * cs - y0 * sn], -1)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        dw += (x * u).sum((0, 1))
    # (a thread adds up some 600 tokens' rows here: 0.42 * 25 roundings more, in squares)
    la_norms.check(g["dwq"], dw, la_norms.DW, "dwq")
    del q, gq, o, g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,d", [(torch.float32, 16), (torch.bfloat16, 128)])
def test_packed_without_tokens(ck, dtype, d):  # noqa: F811
    q, k, v, a, dO, S0, dSf = make((0,), 2, d, d, dtype, seed=5, n=3)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu)
    g = ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu)
    assert ck.device_status() == 0
    assert o.shape == v.shape and torch.equal(S, S0) and torch.equal(g["dS0"], dSf)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_replayed_with_other_offsets(ck, dtype):  # noqa: F811
    """The offsets are read on the device: a captured call follows them."""
    q, k, v, a, dO, S0, dSf = make((700,), 2, 64, 64, dtype, seed=6, n=4)
    cu = torch.tensor([0, 100, 100, 650, 700], dtype=torch.int32, device=DEV)
    run = lambda: (ck.la_fwd_chunked(q, k, v, a, S0=S0, cu_seqlens=cu),  # noqa: E731
                   ck.la_bwd_chunked(q, k, v, a, dO, S0=S0, dS_final=dSf, cu_seqlens=cu))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, S), g = run()
    for other in ([0, 0, 700, 700, 700], [0, 1, 129, 257, 700], [0, 175, 350, 525, 700]):
        cu.copy_(torch.tensor(other, dtype=torch.int32, device=DEV))
        graph.replay()
        (eo, eS), eg = run()
        assert torch.equal(o, eo) and torch.equal(S, eS)
        assert all(torch.equal(g[n], eg[n]) for n in g)
        check_forward(o, S, *la_ref.forward(q, k, v, a, S0, cu), dtype == torch.bfloat16)
    assert ck.device_status() == 0


@pytest.mark.parametrize("d", [16, 64, 128])
def test_results_of_another_type(ck, d):  # noqa: F811
    for dtype, out in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        tc = dtype == torch.bfloat16 and d >= 64
        q, k, v, a, _, S0, _ = make((2, 150), 2, d, d, dtype, seed=7)
        o, S = ck.la_fwd_chunked(q, k, v, a, S0=S0, out_dtype=out)
        assert o.dtype == out
        check_forward(o, S, *la_ref.forward(q, k, v, a, S0), tc)
        y = ck.la_decode_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                              a[:, 0].contiguous(), S1 := S0.clone(), out_dtype=out)
        assert y.dtype == out
        check_forward(y[:, None], S1, *la_ref.forward(*(x[:, :1] for x in (q, k, v, a)), S0), False)
        given = torch.full_like(v, float("nan"), dtype=out)
        ck.la_fwd_chunked(q, k, v, a, S0=S0, out=given)
        assert torch.equal(given, o)
