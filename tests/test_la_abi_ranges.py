"""Sizes and strides of the head-decay attention and the norm whose extents
leave 64 bits are refused on the host (CPU only; fake addresses)."""
import pytest

from test_la_abi import at, lib, norm, normb  # noqa: F401

FAR = {name: (i + 1) << 44 for i, name in enumerate(("oq", "ok"))}
FARB = {name: (i + 1) << 44 for i, name in enumerate(("gq", "gk", "dq", "dk", "dwq", "dwk", "ws"))}


@pytest.mark.parametrize("side", ["qs", "ks"])
def test_strides_whose_extent_wraps_around(lib, side):  # noqa: F811
    n = (1 << 30) + 1
    # 2^30 strides of 2^33 bf16 elements are 2^64 bytes: an extent of one row after the wrap
    for stride in (1 << 33, 1 << 40, 1 << 62, (1 << 62) + 64, (1 << 63) - 64):
        assert norm(lib, n=n, **FAR, **{side: stride}) == -1, stride
        assert normb(lib, n=n, **FARB, wsb=1 << 30, **{side: stride}) == -1, stride
    # one far row is no extent that wraps, and still must not lie in an output
    assert norm(lib, n=2, oq=at(0) + (1 << 30), qs=1 << 29) == -1
    assert normb(lib, n=2, dq=at(0) + (1 << 30), qs=1 << 29) == -1
