"""Open and closed gates of the norm around a block: their values and slopes keep their relative
accuracy, however small they get."""
import pytest
import torch

import norm_ref as ref
from gpu_util import say
from test_gpu_norm import HALF, backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("after", [True, False])
def test_far_gates(act, dtype, after):
    """h = scale n act(z) and dgate = dh scale n slope(z) are products: each factor is within the
    roundings that norm_ref counts, and e^-|z| within |z| 2^-24 of its own size more (the rounded
    argument), so that both are compared with their own size."""
    say(f"gates far from zero {act} {dtype} after {after}")
    d = ref.make(8, 64, dtype, after=after, gate=act, residual=False, before=False, seed=15)
    at = torch.tensor([4.0, 8.0, 12.0, 16.0, 17.5, 20.0, 40.0, 60.0])
    d["gate"] = torch.cat([at, -at]).repeat(4).expand(8, 64).contiguous().to(d["gate"].dtype)
    far = 60 * 2.0 ** -24
    h, _ = forward(d, torch.float32)
    want, _ = ref.forward(d)
    ref.check("h", h, want, want.abs(), ref.FORWARD_EPS + far, HALF[torch.float32])
    out = backward(d, torch.float32)
    # (s (1 - s) of a rounded s loses open gates in float64 too: the slope from e^-|z|)
    z = d["gate"].double()
    small = torch.exp(-z.abs()) / (1 + torch.exp(-z.abs()))
    s, rest = torch.where(z < 0, small, 1 - small), torch.where(z < 0, 1 - small, small)
    slope = s * rest if act == "sigmoid" else s * (1 + z * rest)
    n, _ = ref.forward(dict(d, gate=None, scale=1.0))
    want = d["scale"] * d["dh"].double() * n * slope
    ref.check("dgate", out["dgate"], want, want.abs(), ref.BACKWARD_EPS + far, HALF[torch.float32])
