"""Checks of linear attention in the 2-norm.  Elementwise bounds (linear_ref.slack) add up the
absolute values of all terms, which a result of random signs never comes near; here the roundings
are taken as what they are, independent and of either sign, so that a lost plane, a biased factor
or a wrong gate gradient shows.

A rounding to fp32 is off by at most 2^-24 of its value, 2^-24 / sqrt(3) in the root mean square,
and n of them along a sum whose partial sums stay below the result's size leave sqrt(n) of that.
Counted for 128 x 128 and chunks of 64 tokens, each product of 32 terms as eight roundings and each
of its planes as a product of its own:
  - scores: 4 blocks, 32 roundings; their decays and scale 6;
  - P w: 2 blocks in 3 planes, 48; Z x: 4 blocks in 3 planes, 96; sums and stores 8;
  - Z: 2 blocks in 3 planes and the decay for each chunk that is walked, 49;
  - dot products of the gate gradient: 32."""
import math

import torch

import linear_ref as ref

F64 = torch.float64

# Cases of the gate gradient: lens, H, Hk, dk, dv, decay, gate, with states at both ends or not.
GATES = [
    ([64], 4, 2, 128, 128, "head", "std", False),
    ([2, 0, 65], 4, 2, 128, 128, "head", "std", True),
    ([300, 0, 1, 129], 4, 1, 64, 128, "head", "slow", False),
    ([300, 0, 1, 129], 4, 2, 64, 64, "token", "slow", True),
    ([63, 64, 65, 1, 128], 2, 2, 128, 64, "token", "std", True),
    ([200, 65, 3], 4, 2, 128, 128, "token", "reset", True),
    ([200, 65, 3], 4, 2, 64, 64, "token", "steep", True),
    # in segments
    ([1600], 2, 1, 64, 128, "head", "slow", True),
    ([1600], 2, 1, 128, 128, "token", "slow", True),
    ([0, 30, 1025], 2, 1, 128, 64, "token", "unit", False),
]


def gate_case(dtype, lens, H, Hk, dk, dv, decay, gate, state):
    return ref.make(lens, H, Hk, dk, dv, dtype, decay, gate, state, seed=71)


def walk(d, more=0):
    """Relative 2-norm of the error of an output of inputs d."""
    n = 190 + more + 49 * math.ceil(max(d["lens"]) / 64)
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


def gate_tolerance(d):
    """Relative error of dg.  Its terms are row_t - col_t, dot products of outputs (walk, twice), of
    which row_t is a part of dg_t's own sum and so no larger; the suffix sums, tied at both ends,
    carry them over at most the sequence: sqrt(L) for the values of single tokens.  Summed over the
    tokens for one gate a head such a bridge of L steps leaves L^1.5 / sqrt(12) of a step's error,
    beside at least sqrt(L) of dg_t."""
    L = max(d["lens"])
    more = L / math.sqrt(12) if d["g"].dim() == 1 else math.sqrt(L)
    return walk(d, 32) * math.sqrt(2) * max(more, 1.0)


def gate_gradient_errors(d, got, want):
    """(sequence, error, size) of dg for each sequence, over its tokens and heads; one gate a head:
    over the heads, sequence None."""
    got = got.detach().to("cpu", F64)
    if d["g"].dim() == 1:
        return [(None, *distance(got, want))]
    out = []
    for n, L in enumerate(d["lens"]):
        at = slice(int(d["cu"][n]), int(d["cu"][n]) + L)
        out.append((n, *distance(got[at], want[at])))
    return out


def check_gate_gradient(d, got, want=None):
    want = ref.backward(d)["dg"] if want is None else want
    tol = gate_tolerance(d)
    for n, far, size in gate_gradient_errors(d, got, want):
        if size or far:
            print(f"dg of sequence {n}: {far / size if size else far:.2e} of {tol:.2e}", flush=True)
        assert far <= tol * size, (n, far, size, tol)
