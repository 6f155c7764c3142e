"""The checks of linear_norms reject wrong results: gate gradients of zeros, of the other sign, half
as large again, without the term of the final states, or with one head's values lost, and outputs
of products in two bf16 planes."""
import pytest
import torch

import linear_norms as norms
import linear_ref as ref


def _rejected(d, got, want):
    with pytest.raises(AssertionError):
        norms.check_gate_gradient(d, got, want)


@pytest.mark.parametrize("case", norms.GATES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wrong_gate_gradients_are_rejected(case, dtype):
    d = norms.gate_case(dtype, *case)
    want = ref.backward(d)["dg"]
    assert norms.gate_tolerance(d) < 0.01
    norms.check_gate_gradient(d, want, want)
    for wrong in (0 * want, -want, 1.5 * want, 0.98 * want):
        _rejected(d, wrong, want)
    for h in range(d["H"]):
        wrong = want.clone()
        wrong[..., h] = 0
        _rejected(d, wrong, want)
    if d["dstate_out"] is not None:
        _rejected(d, ref.backward(dict(d, dstate_out=None))["dg"], want)
    if d["state_in"] is not None:
        # S_0's part: the gradient of a call from zero states
        _rejected(d, ref.backward(dict(d, state_in=torch.zeros_like(d["state_in"])))["dg"], want)


def test_two_planes_are_rejected():
    """P w of one chunk with P in two bf16 planes and in three."""
    gen = torch.Generator().manual_seed(1)
    P, w = torch.randn(64, 64, generator=gen), torch.randn(64, 128, generator=gen)
    want = P.double() @ w.double()
    hi = P.bfloat16().float()
    mid = (P - hi).bfloat16().float()
    low = (P - hi - mid).bfloat16().float()
    d = dict(lens=[300])
    norms.check("three planes", (hi.double() + mid.double() + low.double()) @ w.double(), want,
                norms.walk(d))
    with pytest.raises(AssertionError):
        norms.check("two planes", (hi.double() + mid.double()) @ w.double(), want, norms.walk(d))
