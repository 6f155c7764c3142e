"""Infinite scales of the product in 8 bits on the GPU: an infinity of the block sum's sign, not a
NaN, whatever the shape of workgroup and however the blocks go round its groups of waves."""
import pytest
import torch

import product_ref as ref
from gpu_util import say
from test_gpu_product import SHAPES, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [144, 272, 400, 640, 1040])
@pytest.mark.parametrize("M, N", [(5, 270)] + SHAPES)
@pytest.mark.parametrize("which", ["sa", "sw"])
def test_infinite_scales(M, N, K, which):
    say(f"product M {M} N {N} K {K} {which} infinite")
    d = ref.make(M, N, K, seed=K)
    last = d["sa"].shape[1] - 1
    # the last value of a row, 1 in a and never zero in w, is its last block's sum
    a, w = d["a"].float(), d["w"].float()
    a[:, last * 128:] = 0
    a[:, -1] = 1
    w[:, -1] = torch.where(w[:, -1] == 0, 1.0, w[:, -1])
    d["a"], d["w"] = a.to(ref.E4M3), w.to(ref.E4M3)
    clean = {t: run(d, t) for t in (torch.float32, torch.bfloat16)}
    rows, cols = torch.zeros(M, dtype=torch.bool), torch.zeros(N, dtype=torch.bool)
    if which == "sa":
        d["sa"][3, last] = d["sa"][M - 1, last] = float("inf")
        rows[3] = rows[M - 1] = True
        cols[:] = True
    else:
        d["sw"][0, last] = float("inf")
        rows[:] = True
        cols[:128] = True
    hit = (rows[:, None] & cols[None]).cuda()
    want = torch.sign(w[:, -1]).cuda().expand(M, N) * float("inf")
    for t in clean:
        got = run(d, t)
        assert torch.equal(got[hit].float(), want[hit]), t
        assert torch.equal(got[~hit], clean[t][~hit]), t
