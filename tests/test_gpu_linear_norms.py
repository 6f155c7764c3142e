"""Linear attention with a decay for each head on the GPU against float64 in the 2-norm
(linear_norms): gate gradients whose tolerance is far below their own size, and outputs that hold
what fp32 arithmetic leaves."""
import pytest
import torch

import linear_norms as norms
import linear_ref as ref
from gpu_util import say
from test_gpu_linear import backward, dev, prefill

pytestmark = pytest.mark.gpu


def check_outputs(d):
    """Every fp32 output and gradient, the gradients with and without that of the gates."""
    T = int(d["cu"][-1])
    o, s = prefill(d, torch.float32)
    want_o, want_s = ref.forward(d)
    norms.check("o", o[:T], want_o, norms.walk(d))
    norms.check("state_out", s, want_s, norms.walk(d))
    want = ref.backward(d)
    for dg in (True, False):
        out = backward(d, torch.float32, dg=dg)
        for n in ("dq", "dk", "dv", "dstate_in"):
            if n in out:
                norms.check(n, out[n], want[n], norms.walk(d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk, dv, H, Hk", [(128, 128, 4, 2), (64, 64, 3, 3), (64, 128, 4, 1),
                                           (128, 64, 2, 2)])
def test_fp32_outputs_hold_fp32(dtype, dk, dv, H, Hk):
    say(f"fp32 outputs of {dtype} inputs {dk}x{dv} H{H}/{Hk}")
    check_outputs(ref.make([300, 130, 65], H, Hk, dk, dv, dtype, "token", "slow", True, seed=38))


@pytest.mark.parametrize("scale", [1e-20, -1e12])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_far_from_one(scale, dtype):
    """From zero states every value comes from the scores, so that their scale shows."""
    say(f"scale {scale} of {dtype} inputs")
    d = ref.make([64, 300, 7], 4, 2, 128, 128, dtype, "token", "slow", False, seed=39)
    d["scale"] = scale
    check_outputs(d)


@pytest.mark.parametrize("case", norms.GATES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gate_gradient(case, dtype):
    say(f"gate gradient {case} {dtype}")
    d = norms.gate_case(dtype, *case)
    norms.check_gate_gradient(d, backward(d)["dg"])


@pytest.mark.parametrize("decay", ["token", "head"])
def test_gate_gradient_against_differences(decay):
    """Differences of the prefill kernel itself along a direction of gates, in fp32.  Five points
    leave f^(5) h^4 / 30 of the derivative's own size: with h = 2^-5 and gates that move by h times
    a normal number over the few tokens that a memory of std gates spans, below 1e-4.  The roundings
    of the loss, walk(d) of the root sum of squares of its terms, come on top, over h."""
    import gated_delta_rule_100_amd as gdr
    lens, H, d = [130, 20], 4, 64
    case = ref.make(lens, H, 2, d, d, "f32", decay, "std", True, seed=37)
    x = dev(case)
    dg = backward(case, x=x)["dg"].double()
    T, N, h = sum(lens), len(lens), 2.0 ** -5
    o, s = torch.empty(T, H, d, device="cuda"), torch.empty(N, H, d, d, device="cuda")
    terms = []

    def loss(g):
        gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], g, x["cu"], x["state_in"], s, o,
                               scale=case["scale"])
        p, r = o.double() * x["do"].double(), s.double() * x["dstate_out"].double()
        terms.append(float((p.square().sum() + r.square().sum()).sqrt()))
        return float(p.sum() + r.sum())

    gen = torch.Generator(device="cuda").manual_seed(3)
    for i in range(3):
        say(f"differences along gates, {decay}, direction {i}")
        step = torch.randn(x["g"].shape, generator=gen, device="cuda")
        if decay == "head":  # every token of a head moves together: a shorter step
            step = step / 4
        at = {m: loss(x["g"] + m * h * step) for m in (-2, -1, 1, 2)}
        got = (8 * (at[1] - at[-1]) - (at[2] - at[-2])) / (12 * h)
        want = float((dg * step.double()).sum())
        room = 1e-3 * float((dg * step.double()).norm()) + 2 * norms.walk(case) * max(terms) / h
        assert room < 0.05 * float((dg * step.double()).norm())
        assert abs(got - want) < room, (got, want, room)
