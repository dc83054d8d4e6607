"""Refusals of the head-decay linear attention and of the query / key norm:
argument errors are found on the host, before any CUDA call (CPU only)."""
import pytest

P = 1 << 32           # fake device addresses, never dereferenced
STEP = 1 << 24        # room between two tensors
MIS = P + 4
WS = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from delta_rule_linear_ckda_b200 import build as b

    b.build()
    from delta_rule_linear_ckda_b200 import _lib

    return _lib.load()


def at(i):
    return P + i * STEP


def fwd(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), alpha=at(3), S0=None, cu=None, out=at(4), Sf=None, B=1, T=8,
             H=2, dk=16, dv=16, per_head=0, dtype=0, odt=0, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.ckda_la_fwd_chunked(*a.values())


def bwd(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), alpha=at(3), S0=None, cu=None, dO=at(4), dSf=None, dq=at(5),
             dk_=at(6), dv_=at(7), da=at(8), dS0=None, B=1, T=8, H=2, dk=16, dv=16, per_head=0,
             dtype=0, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.ckda_la_bwd_chunked(*a.values())


def step(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), alpha=at(3), S=at(4), out=at(5), B=2, H=2, dk=16, dv=16,
             per_head=0, dtype=1, odt=0, stream=None)
    a.update(kw)
    return lib.ckda_la_decode_step(*a.values())


def norm(lib, **kw):
    a = dict(q=at(0), k=at(1), wq=at(2), wk=at(3), pos=at(4), freq=at(5), oq=at(6), ok=at(7), n=4,
             Hq=2, Hk=1, d=32, rot=16, il=0, norm=1, eps=1e-6, qs=64, ks=32, dtype=1, odt=1,
             stream=None)
    a.update(kw)
    return lib.ckda_qk_norm_rope(*a.values())


def normb(lib, **kw):
    a = dict(q=at(0), k=at(1), wq=at(2), wk=at(3), pos=at(4), freq=at(5), gq=at(6), gk=at(7),
             dq=at(8), dk=at(9), dwq=at(10), dwk=at(11), n=4, Hq=2, Hk=1, d=32, rot=16, il=0, norm=1,
             eps=1e-6, qs=64, ks=32, dtype=1, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.ckda_qk_norm_rope_bwd(*a.values())


def test_forward(lib):
    for name in ("q", "k", "v", "alpha", "out"):
        assert fwd(lib, **{name: None}) == -1, name
        assert fwd(lib, **{name: MIS}) == -3, name
    assert fwd(lib, B=-1) == -1
    assert fwd(lib, T=-1) == -1
    assert fwd(lib, H=0) == -1
    assert fwd(lib, per_head=2) == -1
    assert fwd(lib, dk=48) == -2
    assert fwd(lib, dv=256) == -2
    assert fwd(lib, dtype=2) == -2
    assert fwd(lib, odt=-1) == -2
    assert fwd(lib, H=65536, T=1) == -2
    assert fwd(lib, B=1 << 16, T=1 << 14, H=4) == -2       # tokens times heads beyond 31 bits
    assert fwd(lib, S0=MIS) == -3
    assert fwd(lib, cu=at(9) + 2) == -3
    assert fwd(lib, cu=at(9), B=0, T=5) == -1              # tokens but no sequence
    assert fwd(lib, B=0) == 0
    # overlaps: 8 tokens of 2 heads of 16 channels are 1024 bytes
    assert fwd(lib, out=at(0)) == -1
    assert fwd(lib, out=at(0) + 1008) == -1
    assert fwd(lib, Sf=at(2) + 16) == -1
    assert fwd(lib, S0=at(5), Sf=at(5) + 16) == -1
    assert fwd(lib, out=at(5), S0=at(5)) == -1


def test_backward(lib):
    for name in ("q", "k", "v", "alpha", "dO", "dq", "dk_", "dv_", "da"):
        assert bwd(lib, **{name: None}) == -1, name
        assert bwd(lib, **{name: MIS}) == -3, name
    assert bwd(lib, T=0, per_head=1, da=None) == -1        # [H] is written whatever T
    assert bwd(lib, dk=8) == -2
    assert bwd(lib, dtype=5) == -2
    assert bwd(lib, dq=at(0)) == -1
    assert bwd(lib, dq=at(6) + 512) == -1                  # two outputs
    assert bwd(lib, dS0=at(9), dSf=at(9)) == -1
    assert bwd(lib, B=0) == 0
    need = lib.ckda_la_bwd_workspace_bytes(1, 8, 2, 16, 16, 0, 0, 0)
    assert need > 0
    assert bwd(lib) == -7
    assert bwd(lib, ws=WS, wsb=need - 1) == -7
    assert bwd(lib, ws=WS + 16, wsb=need) == -7
    assert bwd(lib, ws=at(2), wsb=need) == -7
    assert bwd(lib, ws=at(2) - 256, wsb=1 << 30) == -7     # reaches into v
    q = lib.ckda_la_bwd_workspace_bytes
    assert q(1, 8, 2, 16, 48, 0, 0, 0) == -2
    assert q(1, 8, 0, 16, 16, 0, 0, 0) == -1
    assert q(0, 0, 2, 16, 16, 0, 0, 0) == 0
    assert lib.ckda_la_fwd_workspace_bytes(1, 8, 2, 24, 16, 0, 0) == -2


def test_step(lib):
    for name in ("q", "k", "v", "alpha", "S", "out"):
        assert step(lib, **{name: None}) == -1, name
        assert step(lib, **{name: MIS}) == -3, name
    assert step(lib, H=0) == -1
    assert step(lib, dk=24) == -2
    assert step(lib, dtype=3) == -2
    assert step(lib, odt=9) == -2
    assert step(lib, out=at(4)) == -1
    assert step(lib, S=at(2)) == -1
    assert step(lib, B=0) == 0


def test_norm(lib):
    for call, extra in ((norm, ("oq", "ok")), (normb, ("gq", "gk", "dq", "dk"))):
        for name in ("q", "k", "pos", "freq") + extra:
            assert call(lib, **{name: None}) == -1, name
        for name in ("q", "k") + extra:
            assert call(lib, **{name: MIS}) == -3, name
        assert call(lib, wq=at(2) + 2) == -3
        assert call(lib, n=-1) == -1
        assert call(lib, Hq=0, Hk=0) == -1
        assert call(lib, rot=40) == -1
        assert call(lib, rot=12) == -2
        assert call(lib, d=48) == -2
        assert call(lib, norm=2) == -1
        assert call(lib, il=3) == -1
        assert call(lib, eps=-1e-6) == -1
        assert call(lib, eps=float("nan")) == -1
        assert call(lib, eps=float("inf")) == -1
        assert call(lib, qs=63) == -1              # tokens would overlap
        assert call(lib, qs=68) == -3              # rows not 16-byte aligned
        assert call(lib, dtype=4) == -2
        assert call(lib, n=1 << 31) == -2
    assert norm(lib, odt=2) == -2
    assert norm(lib, n=0) == 0
    assert norm(lib, oq=at(1)) == -1               # q_out on k
    assert norm(lib, oq=at(0) + 64) == -1          # shifted by half a row
    assert norm(lib, oq=at(0), qs=128) == -1       # in place of a strided input
    assert norm(lib, oq=at(0), odt=0) == -1        # in place with another type
    assert norm(lib, oq=at(6), ok=at(6)) == -1
    assert normb(lib, dq=at(0)) == -1
    assert normb(lib, dwq=at(11)) == -1
    assert normb(lib, n=0, dwq=None, dwk=None) == 0
    need = lib.ckda_qk_norm_rope_bwd_workspace_bytes(32)
    assert need > 0 and lib.ckda_qk_norm_rope_bwd_workspace_bytes(33) == -2
    assert normb(lib) == -7
    assert normb(lib, ws=WS, wsb=need - 4) == -7
    assert normb(lib, ws=at(8), wsb=need) == -7
