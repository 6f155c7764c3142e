"""The checks of linear_norms reject outputs of products in two bf16 planes."""
import pytest
import torch

import linear_norms as norms


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
