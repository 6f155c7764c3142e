"""Linear attention with a decay for each head at the ends of its range: segment tables in memory,
offsets past 2^31 and strides of 2^24 elements, resets, scales of both signs, empty batches."""
import pytest
import torch

import linear_ref as ref
from gpu_util import say
from test_gpu_linear import HALF, backward, check_backward, check_prefill, dev, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_of_more_sequences_than_a_wave_has_lanes(dtype):
    import gated_delta_rule_100_amd as gdr
    lens = [900, 0, 1, 128, 129] + [200 + 3 * i for i in range(66)] + [640]
    T, N = sum(lens), len(lens)
    assert gdr.gdr_linear_prefill_workspace_bytes(T, N, 2, 64, 64) > 0  # segments, and N > 64
    say(f"{N} sequences in segments {dtype}")
    d = ref.make(lens, 2, 1, 64, 64, dtype, "token", "slow", True, seed=91)
    check_prefill(d, *prefill(d))
    check_backward(d, backward(d))


def test_gradient_of_a_reset_gate_is_zero():
    d = ref.make([300, 65], 3, 3, 64, 128, "bf16", "token", "reset", True, seed=92)
    d["g"][10] = -111.0
    out = backward(d)
    reset = (d["g"] < -110).cuda()
    assert reset.any() and not out["dg"][reset].any()
    check_backward(d, out)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(scale, dtype):
    say(f"scale {scale} {dtype}")
    d = ref.make([130, 7], 4, 2, 64, 128, dtype, "token", "slow", True, seed=93)
    d["scale"] = scale
    check_prefill(d, *prefill(d))
    check_backward(d, backward(d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_on_strided_tokens(dtype):
    say(f"backward on slices of one fused projection {dtype}")
    d = ref.make([90, 40], 4, 2, 64, 128, dtype, seed=94)
    x = dev(d)
    fused = torch.full((130, 2 * 128 + 512 + 16), float("nan"), device="cuda", dtype=x["q"].dtype)
    q, k = fused[:, :128].view(130, 2, 64), fused[:, 128:256].view(130, 2, 64)
    v = fused[:, 256:768].view(130, 4, 128)
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    dense = backward(d, x=x)
    x.update(q=q, k=k, v=v)
    strided = backward(d, x=x)
    assert all(torch.equal(dense[n], strided[n]) for n in dense)


@pytest.mark.parametrize("decay", ["token", "head"])
def test_backward_of_no_tokens(decay):
    d = ref.make([0, 0], 2, 2, 64, 64, "bf16", decay, seed=95)
    out = backward(d)
    assert torch.equal(out["dstate_in"].cpu(), d["dstate_out"])
    assert not out["dg"].any()


def test_strides_of_2_24_elements():
    """Tokens 64 MiB apart (fp32): byte offsets inside a chunk up to 63 * 2^26, and past 2^31
    elements over the batch."""
    import gated_delta_rule_100_amd as gdr
    say("prefill with strides of 2^24 elements")
    d = ref.make([130], 2, 2, 64, 64, "f32", seed=96)
    x = dev(d)
    wide = torch.empty(130, 1 << 24, device="cuda")
    q, k, v = (wide[:, at:at + 128].view(130, 2, 64) for at in (0, 128, (1 << 24) - 128))
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    dense = prefill(d, x=x)
    x.update(q=q, k=k, v=v)
    strided = prefill(d, x=x)
    assert torch.equal(dense[0], strided[0]) and torch.equal(dense[1], strided[1])
    out = backward(d, x=x)
    check_backward(d, out)
    w = torch.as_strided(wide, (2, 2, 64), ((1 << 24) + 4, 64, 1))
    with pytest.raises(gdr.GdrError, match="2\\^24"):
        gdr.gdr_linear_prefill(w, x["k"][:2], x["v"][:2], x["g"][:2], x["cu"] * 0, None, None,
                               torch.empty(2, 2, 64, device="cuda"))


def test_more_than_2_31_elements():
    """131272 tokens of 128 heads: the last sequence lies behind element 2^31 of every tensor."""
    import gated_delta_rule_100_amd as gdr
    H, D, first, last = 128, 128, 65, 70
    T = (1 << 31) // (H * D) + 130 + last
    say(f"prefill and backward of {T} tokens, {H} heads")
    d = ref.make([last], H, H, D, D, "bf16", "token", "slow", False, seed=97)
    e = ref.make([first], H, H, D, D, "bf16", "token", "slow", False, seed=98)
    x = {n: torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16) for n in ("q", "k", "v", "do")}
    g = torch.zeros(T, H, device="cuda")
    for n in x:
        x[n][:first].copy_(e[n])
        x[n][T - last:].copy_(d[n])
    g[:first].copy_(e["g"])
    g[T - last:].copy_(d["g"])
    cu = torch.tensor([0, first, T - last, T], dtype=torch.int32, device="cuda")
    o = torch.full((T, H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    s = torch.empty(3, H, D, D, device="cuda")
    gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], g, cu, None, s, o, scale=d["scale"])
    torch.cuda.synchronize()
    for c, at, n in ((e, slice(0, first), 0), (d, slice(T - last, T), 2)):
        check_prefill(c, o[at], s[n:n + 1])
    assert not o[first:T - last].any() and not s[1].any()
    dq, dk, dv = (torch.full_like(o, float("nan")) for _ in range(3))
    dg = torch.full_like(g, float("nan"))
    gdr.gdr_linear_backward(x["q"], x["k"], x["v"], g, cu, None, x["do"], None, dq, dk, dv, dg=dg,
                            scale=d["scale"])
    torch.cuda.synchronize()
    for c, at in ((e, slice(0, first)), (d, slice(T - last, T))):
        c["dstate_out"] = None
        check_backward(c, dict(dq=dq[at], dk=dk[at], dv=dv[at], dg=dg[at]))
    for t in (dq, dk, dv, dg):
        assert not t[first:T - last].any()


def test_decode_of_more_than_2_31_state_elements():
    import gated_delta_rule_100_amd as gdr
    N, H, D = 1030, 128, 128
    say(f"decode of {N} x {H} states")
    d = ref.make([1] * 2, H, H, D, D, "bf16", "token", "std", True, seed=99)
    q, k, v = (torch.zeros(N, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    g = torch.zeros(N, H, device="cuda")
    s = torch.zeros(N, H, D, D, device="cuda")
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (s, "state_in")):
        t[0].copy_(d[n][0])
        t[-1].copy_(d[n][1])
    o = torch.full((N, H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    gdr.gdr_linear_decode(q, k, v, g, s, o, scale=d["scale"])
    torch.cuda.synchronize()
    want_o, want_s = ref.forward(d)
    b = ref.bounds(d)
    ref.check("o", o[[0, N - 1]], want_o, b["o"], 136 * 2.0 ** -24, HALF[o.dtype])
    ref.check("state", s[[0, N - 1]], want_s, b["state_out"], 136 * 2.0 ** -24)
    assert not o[1:-1].any() and not s[1:-1].any()
