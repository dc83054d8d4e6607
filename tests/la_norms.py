"""Relative 2-norm bounds for head-decay linear attention and the norm's weight
gradients, beside the elementwise worst cases of la_ref: those grow with the
sums' absolute values and let a long sum lose a whole term.

Rounding to bf16 is off by 1.66e-3 of the value in the mean square: uniform in
half a step of 2^-7, over mantissas spread logarithmically, sqrt(0.541 / 3)
2^-8.  Independent roundings add in squares.

  LOW  outputs rounded to bf16 (out, dq, dk, dv on the tensor cores): the result's
       own rounding and that of one operand of each of the two products that it
       is the sum of, sqrt(2) 1.66e-3 = 2.35e-3; half as much again is allowed.
  ROUND  the rounding of the result alone, of a form that is fp32 up to there.
  FULL what keeps fp32 accuracy (S_final, dS0, dalpha, and every result of fp32
       inputs), with decays that differ from token to token: some 35 products on
       a weight's way through a chunk and 40 sums are independent roundings of
       0.42 2^-24, 4 2^-24 in all, and the tensor cores' sums cut off instead of
       rounding, once for each of the 8 steps of a product, half a unit each:
       8 2^-24 = 4.8e-7 together.  Twice that is allowed.  A split into two bf16
       terms instead of three leaves 1e-6 to 2.5e-6.
  DW   a weight's gradient: (d + 24 + 16) 2^-24 = 1e-5 for d = 128, the roundings
       of a row's norm and turn and of some 16 rows in a thread's sum.
"""
import torch

LOW = 3.5e-3
ROUND = 2.0e-3
FULL = 16 * 2.0 ** -24
DW = 1.0e-5


def off(got, ref, dims=None):
    """|got - ref| / |ref| in 2-norm, over ``dims`` (all of them when None); 0 where both are 0."""
    got, ref = got.detach().cpu().double(), ref.detach().cpu().double()
    assert got.shape == ref.shape
    dims = tuple(range(ref.dim())) if dims is None else dims
    e, r = ((x * x).sum(dims).sqrt() for x in (got - ref, ref))
    return torch.where(e == 0, e, e / r)


def near(got, ref, bound, heads=None):
    """The whole tensor is within ``bound`` and, with the dimension of the heads given, twice
    that for every head by itself, if a head has 32 elements or more.  The error follows the
    sums' terms, not the result: of n results that are sums of random signs, normal with
    deviation s, the norm is below half of s sqrt(n) with the chance that chi^2 of n degrees
    is below n / 4, 1e-6 for n = 32; a single one is below a half in 38 cases of 100, and below
    a tenth in 8."""
    if ref.numel() == 0:
        return True
    ok = bool(off(got, ref) <= bound)
    if heads is not None and ref.numel() // ref.shape[heads] >= 32:
        dims = tuple(i for i in range(ref.dim()) if i != heads % ref.dim())
        ok = ok and bool((off(got, ref, dims) <= 2 * bound).all())
    return ok


def check(got, ref, bound, name="", heads=None):
    assert near(got, ref, bound, heads), (name, float(off(got, ref)), bound)
