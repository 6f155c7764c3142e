"""Linear attention with a decay for each head on the GPU against the float64
quadratic form, elementwise within the rounding bound of linear_ref.slack."""
import pytest
import torch

import linear_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def dev(d):
    return {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in d.items()}


def prefill(d, out_dtype=None, state_out=True, x=None, workspace=None, stream=None):
    import gated_delta_rule_100_amd as gdr
    x = x or dev(d)
    T, N = x["q"].shape[0], len(d["lens"])
    o = torch.full((T, d["H"], d["dv"]), float("nan"), device="cuda",
                   dtype=out_dtype or x["q"].dtype)
    s = torch.full((N, d["H"], d["dv"], d["dk"]), float("nan"), device="cuda") if state_out else None
    gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], s, o,
                           scale=d["scale"], workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return o, s


def check_prefill(d, o, s, half=None):
    T = int(d["cu"][-1])
    want_o, want_s = ref.forward(d)
    b, eps = ref.bounds(d), ref.slack(d)
    ref.check("o", o[:T], want_o, b["o"], eps, HALF[o.dtype])
    if s is not None:
        ref.check("state_out", s, want_s, b["state_out"], eps, 2.0 ** -24)


# long enough to be cut into segments; one of them starts or ends on a segment's edge
LONG = [[1100, 0, 513, 1, 1024], [1600], [0, 30, 1025]]
LENS = [[1], [64], [2, 0, 65], [63, 64, 65, 1, 128], [300, 0, 1, 129]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk, dv, H, Hk", [(64, 64, 3, 3), (128, 128, 4, 2), (64, 128, 4, 1),
                                           (128, 64, 2, 2)])
def test_prefill(lens, dtype, dk, dv, H, Hk):
    for decay, gate, state in (("token", "slow", True), ("head", "std", False)):
        say(f"prefill {lens} {dtype} {dk}x{dv} H{H}/{Hk} {decay} {gate}")
        d = ref.make(lens, H, Hk, dk, dv, dtype, decay, gate, state, seed=11)
        check_prefill(d, *prefill(d))


@pytest.mark.parametrize("lens", LONG)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk, dv, decay, gate, state", [(128, 128, "token", "slow", True),
                                                        (64, 128, "head", "slow", False),
                                                        (128, 64, "token", "unit", True)])
def test_prefill_in_segments(lens, dtype, dk, dv, decay, gate, state):
    say(f"prefill {lens} {dtype} {dk}x{dv} {decay} {gate}")
    d = ref.make(lens, 2, 1, dk, dv, dtype, decay, gate, state, seed=19)
    o, s = prefill(d)
    check_prefill(d, o, s)
    assert torch.equal(o, prefill(d, state_out=False)[0])


def test_many_sequences_in_segments():
    """More sequences than the kernels form a segment table for by themselves."""
    lens = [1, 0, 700] + [3, 70] * 35 + [650]
    say(f"prefill and backward of {len(lens)} sequences, some in segments")
    d = ref.make(lens, 2, 2, 64, 64, "bf16", "token", "slow", True, seed=20)
    check_prefill(d, *prefill(d))
    check_backward(d, backward(d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["unit", "std", "steep", "reset"])
def test_prefill_gates(dtype, gate):
    say(f"prefill gates {gate} {dtype}")
    d = ref.make([200, 65, 3], 4, 2, 128, 128, dtype, "token", gate, True, seed=12)
    check_prefill(d, *prefill(d, torch.float32))
    # every token resets: only its own key and value remain
    d["g"] = torch.full_like(d["g"], float("-inf"))
    check_prefill(d, *prefill(d, torch.float32))


def test_prefill_bf16_output_is_the_rounded_fp32_output():
    d = ref.make([150, 70], 4, 4, 128, 128, seed=13)
    o32, s32 = prefill(d, torch.float32)
    o16, s16 = prefill(d, torch.bfloat16)
    assert torch.equal(o32.to(torch.bfloat16), o16) and torch.equal(s32, s16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_rows_behind_the_last_sequence(dtype):
    say(f"prefill with NaN rows behind the last sequence {dtype}")
    d = ref.make([70, 33], 4, 2, 64, 128, dtype, seed=14, pad=37)
    o, s = prefill(d)
    assert torch.isnan(o[103:]).all()
    check_prefill(d, o, s)


def test_prefill_other_sequences_values_stay_theirs():
    say("prefill, one sequence of NaN and inf between two others")
    d = ref.make([70, 50, 33], 4, 2, 128, 64, seed=15)
    clean, sclean = prefill(d)
    for n in ("q", "k", "v"):
        d[n][70:120] = float("nan")
    d["v"][75] = float("inf")
    o, s = prefill(d)
    assert torch.equal(o[:70], clean[:70]) and torch.equal(o[120:], clean[120:])
    assert torch.equal(s[0], sclean[0]) and torch.equal(s[2], sclean[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_strided_tokens(dtype):
    say(f"prefill on slices of one fused projection {dtype}")
    d = ref.make([90, 40], 4, 2, 64, 128, dtype, seed=16)
    x = dev(d)
    T, w = 130, 2 * 2 * 64 + 4 * 128 + 16
    fused = torch.full((T, w), float("nan"), device="cuda", dtype=x["q"].dtype)
    q, k = fused[:, :128].view(T, 2, 64), fused[:, 128:256].view(T, 2, 64)
    v = fused[:, 256:768].view(T, 4, 128)
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    dense = prefill(d, x=x)
    x.update(q=q, k=k, v=v)
    strided = prefill(d, x=x)
    assert torch.equal(dense[0], strided[0]) and torch.equal(dense[1], strided[1])


def test_prefill_state_in_place_and_without_state_out():
    import gated_delta_rule_100_amd as gdr
    d = ref.make([130, 0, 5], 4, 4, 128, 128, seed=17)
    x = dev(d)
    o, s = prefill(d, x=x)
    o2, _ = prefill(d, x=x, state_out=False)
    assert torch.equal(o, o2)
    state = x["state_in"].clone()
    gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], state, state, o2,
                           scale=d["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, state)
    assert torch.equal(state[1], x["state_in"][1])  # the empty sequence


def test_prefill_of_no_tokens():
    d = ref.make([0, 0], 2, 2, 64, 64, seed=18)
    o, s = prefill(d)
    assert o.numel() == 0 and torch.equal(s.cpu(), d["state_in"])
    d["state_in"] = None
    _, s = prefill(d)
    assert not s.any()


@pytest.mark.parametrize("N, H, Hk, dk, dv", [(1, 1, 1, 64, 64), (3, 16, 8, 128, 64),
                                              (5, 6, 2, 64, 128), (33, 4, 4, 128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_decode(N, H, Hk, dk, dv, dtype, decay):
    import gated_delta_rule_100_amd as gdr
    say(f"decode N{N} H{H}/{Hk} {dk}x{dv} {dtype} {decay}")
    d = ref.make([1] * N, H, Hk, dk, dv, dtype, decay, "std", True, seed=21)
    x = dev(d)
    s = x["state_in"].clone()
    o = torch.empty(N, H, dv, device="cuda", dtype=x["q"].dtype)
    gdr.gdr_linear_decode(x["q"], x["k"], x["v"], x["g"], s, o, scale=d["scale"])
    torch.cuda.synchronize()
    want_o, want_s = ref.forward(d)
    b = ref.bounds(d)
    # fp32 throughout: alpha (2 steps), a product and a sum, and dk terms of the output
    eps = (dk + 8) * 2.0 ** -24
    ref.check("o", o, want_o, b["o"], eps, HALF[o.dtype])
    ref.check("state", s, want_s, b["state_out"], eps)


def test_decode_reset_and_strided_tokens():
    import gated_delta_rule_100_amd as gdr
    N, H, Hk = 7, 4, 2
    d = ref.make([1] * N, H, Hk, 128, 128, "bf16", "token", "std", True, seed=22)
    d["g"][::2] = float("-inf")
    x = dev(d)
    wide = torch.full((N, 2 * 256 + 512 + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    q, k = wide[:, :256].view(N, Hk, 128), wide[:, 256:512].view(N, Hk, 128)
    v = wide[:, 512:1024].view(N, H, 128)
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    s = x["state_in"].clone()
    o = torch.empty(N, H, 128, device="cuda")
    gdr.gdr_linear_decode(q, k, v, x["g"], s, o, scale=d["scale"])
    torch.cuda.synchronize()
    want_o, want_s = ref.forward(d)
    b = ref.bounds(d)
    ref.check("o", o, want_o, b["o"], 136 * 2.0 ** -24, 2.0 ** -24)
    ref.check("state", s, want_s, b["state_out"], 136 * 2.0 ** -24)


def backward(d, grad_dtype=None, x=None, dg=True, workspace=None, stream=None):
    import gated_delta_rule_100_amd as gdr
    x = x or dev(d)
    gd = grad_dtype or x["q"].dtype
    nan = float("nan")
    out = {n: torch.full(x[n[1:]].shape, nan, device="cuda", dtype=gd) for n in ("dq", "dk", "dv")}
    if dg:
        out["dg"] = torch.full(x["g"].shape, nan, device="cuda")
    if x["state_in"] is not None:
        out["dstate_in"] = torch.full(x["state_in"].shape, nan, device="cuda")
    gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], x["do"],
                            x["dstate_out"], out["dq"], out["dk"], out["dv"], dg=out.get("dg"),
                            dstate_in=out.get("dstate_in"), scale=d["scale"],
                            workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out


def check_backward(d, out):
    want, b, eps = ref.backward(d), ref.bounds(d), ref.slack(d)
    T = int(d["cu"][-1])
    for n, got in out.items():
        if n in ("dq", "dk", "dv") or (n == "dg" and d["g"].dim() == 2):
            got = got[:T]
        e = eps
        if n == "dg":  # and the suffix sum's own roundings
            e += (max(d["lens"]) + T * (d["g"].dim() == 1)) * 2.0 ** -24
        ref.check(n, got, want[n], b[n], e, HALF[got.dtype])


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk, dv, H, Hk", [(64, 64, 3, 3), (128, 128, 4, 2), (64, 128, 4, 1),
                                           (128, 64, 2, 2)])
def test_backward(lens, dtype, dk, dv, H, Hk):
    for decay, gate, state in (("token", "slow", True), ("head", "std", False)):
        say(f"backward {lens} {dtype} {dk}x{dv} H{H}/{Hk} {decay} {gate}")
        d = ref.make(lens, H, Hk, dk, dv, dtype, decay, gate, state, seed=31)
        check_backward(d, backward(d))


@pytest.mark.parametrize("lens", LONG)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk, dv, decay, gate, state", [(128, 128, "token", "slow", True),
                                                        (64, 128, "head", "slow", False),
                                                        (128, 64, "token", "unit", True)])
def test_backward_in_segments(lens, dtype, dk, dv, decay, gate, state):
    say(f"backward {lens} {dtype} {dk}x{dv} {decay} {gate}")
    d = ref.make(lens, 2, 1, dk, dv, dtype, decay, gate, state, seed=36)
    check_backward(d, backward(d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["unit", "std", "steep", "reset"])
def test_backward_gates(dtype, gate):
    say(f"backward gates {gate} {dtype}")
    d = ref.make([200, 65, 3], 4, 2, 128, 128, dtype, "token", gate, True, seed=32)
    out = backward(d, torch.float32)
    check_backward(d, out)
    # without dg another kernel forms dq and dv (fewer planes): the same bound, not the same bits
    check_backward(d, backward(d, torch.float32, dg=False))


@pytest.mark.parametrize("state_in, dstate_out", [(True, False), (False, True)])
def test_backward_with_one_of_the_states(state_in, dstate_out):
    say(f"backward state_in {state_in} dstate_out {dstate_out}")
    d = ref.make([100, 1], 4, 2, 64, 128, "bf16", "token", "slow", True, seed=33)
    if not state_in:
        d["state_in"] = None
    if not dstate_out:
        d["dstate_out"] = None
    check_backward(d, backward(d))


@pytest.mark.parametrize("decay", ["token", "head"])
def test_backward_rows_behind_the_last_sequence(decay):
    say(f"backward with NaN rows behind the last sequence {decay}")
    d = ref.make([70, 33], 4, 2, 64, 128, "bf16", decay, seed=34, pad=37)
    out = backward(d)
    for n in ("dq", "dk", "dv") + (("dg",) if decay == "token" else ()):
        assert torch.isnan(out[n][103:]).all(), n
    check_backward(d, out)


def test_backward_against_differences():
    """Directional derivatives of the prefill kernel itself, in fp32."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make([130, 20], 4, 2, 64, 64, "f32", "token", "std", True, seed=35)
    x = dev(d)
    grads = backward(d, x=x)
    gen = torch.Generator(device="cuda").manual_seed(2)
    eps = 2.0 ** -7

    def loss(y):
        o = torch.empty(150, 4, 64, device="cuda")
        s = torch.empty(2, 4, 64, 64, device="cuda")
        gdr.gdr_linear_prefill(y["q"], y["k"], y["v"], y["g"], y["cu"], y["state_in"], s, o,
                               scale=d["scale"])
        return float((o.double() * x["do"].double()).sum() +
                     (s.double() * x["dstate_out"].double()).sum())

    for name in ("q", "k", "v", "state_in"):
        # the loss is linear in each of these: no truncation error, and rounding of the outputs
        # (2^-24 of terms whose absolute sum bounds the loss) over 2 eps
        step = torch.randn(x[name].shape, generator=gen, device="cuda")
        hi = loss(dict(x, **{name: x[name] + eps * step}))
        lo = loss(dict(x, **{name: x[name] - eps * step}))
        want = float((grads["d" + name].double() * step.double()).sum())
        b, o, s = ref.bounds(d), *ref.forward(d, absolute=True)
        room = float((o * d["do"].double().abs()).sum() + (s * d["dstate_out"].double().abs()).sum())
        # independent roundings of ~10^5 outputs: far below their worst case sum, which would be
        # slack * room / eps; a hundredth of it still shows any wrong term
        assert abs((hi - lo) / (2 * eps) - want) < 0.01 * ref.slack(d) * room / eps, name
        del b


def test_decode_continues_a_prompt():
    """A prompt, then its next tokens one at a time, against the prompt with all of them."""
    import gated_delta_rule_100_amd as gdr
    N, H, Hk, more = 3, 4, 2, 5
    lens = [70, 64, 9]
    full = ref.make([n + more for n in lens], H, Hk, 128, 64, "bf16", "token", "slow", True, seed=41)
    x = dev(full)
    cu = full["cu"].tolist()
    head = torch.cat([torch.arange(cu[n], cu[n] + lens[n]) for n in range(N)]).cuda()
    y = dict(x, cu=torch.tensor([0, 70, 134, 143], dtype=torch.int32, device="cuda"))
    for n in ("q", "k", "v", "g"):
        y[n] = x[n][head].contiguous()
    _, state = prefill(dict(full, lens=lens), x=y)
    outs = []
    for j in range(more):
        at = torch.tensor([cu[n] + lens[n] + j for n in range(N)], device="cuda")
        o = torch.empty(N, H, 64, device="cuda")
        gdr.gdr_linear_decode(*(x[m][at].contiguous() for m in ("q", "k", "v", "g")), state, o,
                              scale=full["scale"])
        outs.append(o)
    torch.cuda.synchronize()
    want_o, want_s = ref.forward(full)
    b, eps = ref.bounds(full), ref.slack(full) + more * 136 * 2.0 ** -24
    for j in range(more):
        at = [cu[n] + lens[n] + j for n in range(N)]
        ref.check(f"o{j}", outs[j], want_o[at], b["o"][at], eps)
    ref.check("state", state, want_s, b["state_out"], eps)


@pytest.mark.parametrize("what", ["prefill", "backward"])
def test_repeated_calls_agree_bit_for_bit(what):
    d = ref.make([300, 64, 1], 4, 2, 128, 128, seed=42)
    x = dev(d)
    run = (lambda: dict(zip("os", prefill(d, x=x)))) if what == "prefill" else (lambda: backward(d, x=x))
    first = run()
    for _ in range(3):
        again = run()
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_calls_on_three_streams():
    import gated_delta_rule_100_amd as gdr
    cases = [ref.make([500, 64], 4, 2, 128, 128, seed=51), ref.make([333], 4, 4, 64, 64, seed=52)]
    xs = [dev(d) for d in cases]
    want_p = [prefill(d, x=x) for d, x in zip(cases, xs)]
    want_b = backward(cases[0], x=xs[0])
    streams = [torch.cuda.Stream() for _ in range(3)]
    o = [torch.empty_like(w[0]) for w in want_p]
    s = [torch.empty_like(w[1]) for w in want_p]
    b = {n: torch.empty_like(t) for n, t in want_b.items()}
    torch.cuda.synchronize()
    for i in range(2):
        x = xs[i]
        gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], s[i], o[i],
                               scale=cases[i]["scale"], stream=streams[i])
    x = xs[0]
    gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], x["do"],
                            x["dstate_out"], b["dq"], b["dk"], b["dv"], dg=b["dg"],
                            dstate_in=b["dstate_in"], scale=cases[0]["scale"], stream=streams[2])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(o[i], want_p[i][0]) and torch.equal(s[i], want_p[i][1])
    assert all(torch.equal(b[n], want_b[n]) for n in b)


def test_in_a_graph():
    """Prompt, gradient and decode step captured together, replayed with new inputs."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make([200, 64, 0, 7], 4, 2, 128, 128, "bf16", "head", "std", seed=53)
    x = dev(d)
    ws_f = torch.empty(max(1, gdr.gdr_linear_prefill_workspace_bytes(271, 4, 4, 128, 128)),
                       dtype=torch.uint8, device="cuda")
    ws_b = torch.empty(gdr.gdr_linear_backward_workspace_bytes(271, 4, 4, 2, 128, 128),
                       dtype=torch.uint8, device="cuda")
    o, s = torch.empty(271, 4, 128, device="cuda"), torch.empty(4, 4, 128, 128, device="cuda")
    od = torch.empty(4, 4, 128, device="cuda")
    b = {n: torch.empty_like(x[n[1:]]) for n in ("dq", "dk", "dv", "dg", "dstate_in")}

    def step(stream=None):
        gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], s, o,
                               scale=d["scale"], workspace=ws_f, stream=stream)
        gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], x["do"],
                                x["dstate_out"], b["dq"], b["dk"], b["dv"], dg=b["dg"],
                                dstate_in=b["dstate_in"], scale=d["scale"], workspace=ws_b,
                                stream=stream)
        gdr.gdr_linear_decode(x["q"][:4], x["k"][:4], x["v"][:4], x["g"], s, od,
                              scale=d["scale"], stream=stream)

    v0 = x["v"].clone()
    outs, want = [o, s, od, *b.values()], []
    for f in (1.0, -0.5):
        x["v"].copy_((f * v0.float()).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    torch.cuda.synchronize()
    for r in range(4):
        x["v"].copy_(((1.0, -0.5)[r % 2] * v0.float()).to(torch.bfloat16))
        for t in outs:
            t.fill_(float("nan"))
        junk = torch.full((1 << 20,), float(r), device="cuda") * 2.0
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(t, w) for t, w in zip(outs, want[r % 2])), r
