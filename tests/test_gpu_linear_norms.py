"""Linear attention with a decay for each head on the GPU against float64 in the 2-norm
(linear_norms): fp32 outputs hold what fp32 arithmetic leaves."""
import pytest
import torch

import linear_norms as norms
import linear_ref as ref
from gpu_util import say
from test_gpu_linear import backward, prefill

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
