"""Checks of linear attention in the 2-norm.  Elementwise bounds (linear_ref.slack) add up the
absolute values of all terms, which a result of random signs never comes near; here the roundings
are taken as what they are, independent and of either sign, so that a lost plane or a biased
factor shows.

A rounding to fp32 is off by at most 2^-24 of its value, 2^-24 / sqrt(3) in the root mean square,
and n of them along a sum whose partial sums stay below the result's size leave sqrt(n) of that.
Counted for 128 x 128 and chunks of 64 tokens, each product of 32 terms as eight roundings and each
of its planes as a product of its own:
  - scores: 4 blocks, 32 roundings; their decays and scale 6;
  - P w: 2 blocks in 3 planes, 48; Z x: 4 blocks in 3 planes, 96; sums and stores 8;
  - Z: 2 blocks in 3 planes and the decay for each chunk that is walked, 49."""
import math

import torch

F64 = torch.float64


def walk(d):
    """Relative 2-norm of the error of an output of inputs d."""
    n = 190 + 49 * math.ceil(max(d["lens"]) / 64)
    return math.sqrt(n / 3) * 2.0 ** -24


def distance(got, want):
    """2-norms of the difference and of the wanted values."""
    got, want = got.detach().to("cpu", F64), want.detach().cpu()
    assert got.shape == want.shape
    return float((got - want).norm()), float(want.norm())


def check(name, got, want, tol):
    far, size = distance(got, want)
    print(f"{name}: {far / size if size else far:.2e} of {tol:.2e}", flush=True)
    assert far <= tol * size, (name, far / size if size else far, tol)
