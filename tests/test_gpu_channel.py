"""The recurrence with a decay for each channel on the GPU against float64, elementwise within
channel_ref's bounds."""
import pytest
import torch

import channel_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

FORMS = [("log", False), ("log", True), ("logit", False), ("logit", True)]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]
RAGGED = [301, 64, 0, 1, 127, 130, 2]


def cuda(d):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in d.items()}


def form(d):
    return dict(gate=d["gate"], complement=d["complement"])


def nan_like(t, *shape):
    return torch.full(shape or t.shape, float("nan"), dtype=t.dtype, device="cuda")


def forward(d, x=None, **kw):
    """h and state_out of the prefill, into buffers of NaN."""
    import gated_delta_rule_100_amd as gdr
    x = x or cuda(d)
    h, out = nan_like(x["x"], *x["x"].shape), torch.full((len(d["lens"]), d["D"]), float("nan"),
                                                        device="cuda")
    gdr.gdr_channel_prefill(x["x"], x["g"], x["cu"], x["state_in"], out, h, **form(d), **kw)
    torch.cuda.synchronize()
    return h, out


def backward(d, h, x=None, **kw):
    import gated_delta_rule_100_amd as gdr
    x = x or cuda(d)
    got = dict(dx=nan_like(h), dg=nan_like(x["g"], *x["g"].shape),
               dstate_in=torch.full((len(d["lens"]), d["D"]), float("nan"), device="cuda"))
    gdr.gdr_channel_backward(x["x"] if d["complement"] else None, x["g"], h, x["cu"], x["state_in"],
                             x["dh"], x["dstate_out"], got["dx"], got["dg"],
                             dstate_in=got["dstate_in"], **form(d), **kw)
    torch.cuda.synchronize()
    return got


def check_all(d):
    T = sum(d["lens"])
    want_h, want_s = ref.forward(d)
    eh, es = ref.forward_bounds(d)
    h, out = forward(d)
    ref.check("h", h[:T], want_h, eh)
    ref.check("state_out", out, want_s, es)
    got = backward(d, h)
    want, bounds = ref.backward(d, h.cpu())
    for n in got:
        ref.check(n, got[n][:T] if n != "dstate_in" else got[n], want[n], bounds[n])
    for t in (h, got["dx"], got["dg"]):
        assert torch.isnan(t[T:]).all()  # rows behind the last sequence
    return h, out, got


@pytest.mark.parametrize("gate, complement", FORMS)
@pytest.mark.parametrize("dtype, gdtype", TYPES)
@pytest.mark.parametrize("D", [136, 77])
def test_forms(gate, complement, dtype, gdtype, D):
    say(f"channel {gate} {complement} {dtype} {gdtype} D {D}")
    check_all(ref.make(RAGGED, D, gate, complement, dtype, gdtype, seed=D, pad=37))


@pytest.mark.parametrize("D", [1, 7, 8, 64, 65, 120, 128, 129, 256, 264])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(D, dtype):
    say(f"channel D {D} {dtype}")
    check_all(ref.make([70, 200], D, "logit", True, dtype, dtype, seed=D))


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [63], [64], [65], [127], [128], [129], [2048],
                                  [2049], [0, 0, 5], [5, 0, 0], [128, 128, 0, 128], [1] * 300,
                                  [0] * 70 + [3] + [0] * 200 + [130] + [0] * 5])
@pytest.mark.parametrize("state", [True, False])
def test_lengths(lens, state):
    say(f"channel lens {lens[:4]}... state {state}")
    check_all(ref.make(lens, 16, "log", False, "bf16", "f32", state=state, seed=len(lens)))
    check_all(ref.make(lens, 9, "logit", True, "f32", "f32", state=state, seed=1))


@pytest.mark.parametrize("kind", ["slow", "steep", "unit", "reset"])
@pytest.mark.parametrize("gate, complement", FORMS)
def test_decays(kind, gate, complement):
    say(f"channel {kind} {gate} {complement}")
    check_all(ref.make([700, 3, 260], 24, gate, complement, "f32", "f32", kind=kind, seed=5))


@pytest.mark.parametrize("D, gate, dtype", [(8, "log", "bf16"), (40, "logit", "f32"),
                                            (3, "log", "f32"), (264, "log", "bf16")])
def test_many_tiles(D, gate, dtype):
    """Sequences over many tiles and blocks of tiles, one ending inside them."""
    say(f"channel many tiles D {D}")
    check_all(ref.make([9000, 1, 6155], D, gate, False, dtype, dtype, kind="slow", seed=6))


def test_constant_decays_close_to_one():
    """A decay of e^-1e-4 at every token: its rounding does not add up over 20000 tokens."""
    d = ref.make([20000], 8, "log", False, "f32", "f32", seed=7)
    d["g"] = torch.full_like(d["g"], -1e-4)
    d["x"] = d["x"].abs()
    want, _ = ref.forward(d)
    h, _ = forward(d)
    err = ((h.cpu().double() - want).norm() / want.norm()).item()
    # a unit in the last place (2^-24) of the decay of 8 tokens, the same one each time, over a
    # reach of 1e4 tokens, and what the 8 tokens themselves leave
    assert err < 1e4 / 8 * 2.0 ** -24 + 16 * 2.0 ** -24, err


def test_gradient_of_zero_outside_operands():
    """No dstate_out, no states, x left out."""
    d = ref.make([100, 30], 32, "log", False, "bf16", "f32", state=False, seed=8)
    check_all(d)


def test_rows_of_wider_tensors_and_in_place():
    import gated_delta_rule_100_amd as gdr
    for D, wide, off in ((64, 208, 104), (33, 100, 40)):
        d = ref.make(RAGGED, D, "logit", True, "bf16", "bf16", seed=9)
        x = cuda(d)
        h, out = forward(d)
        w = torch.full((h.shape[0], wide), float("nan"), dtype=torch.bfloat16, device="cuda")
        sx, sg = w[:, :D], w[:, off:off + D]
        sx.copy_(x["x"])
        sg.copy_(x["g"])
        h2, out2 = forward(d, dict(x, x=sx, g=sg))
        assert torch.equal(h, h2) and torch.equal(out, out2)
        one, two = backward(d, h), backward(d, h, dict(x, x=sx, g=sg))
        assert all(torch.equal(one[n], two[n]) for n in one)
        # in place: h over x, state_out over state_in
        gdr.gdr_channel_prefill(x["x"], x["g"], x["cu"], x["state_in"], x["state_in"], x["x"],
                                **form(d))
        torch.cuda.synchronize()
        assert torch.equal(x["x"], h) and torch.equal(x["state_in"], out)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinities_stay_in_their_sequence_and_channel(value):
    lens = [200, 90, 4000, 333]
    d = ref.make(lens, 24, "log", False, "f32", "f32", seed=10)
    h, out = forward(d)
    back = backward(d, h)
    for n, t, c in ((0, 5, 3), (1, 89, 23), (2, 2500, 0)):
        at = sum(lens[:n]) + t
        e = dict(d, x=d["x"].clone(), dh=d["dh"].clone())
        e["x"][at, c] = value
        e["dh"][at, c] = value
        h2, out2 = forward(e)
        same = torch.ones_like(h, dtype=torch.bool)
        same[at:sum(lens[:n + 1]), c] = False
        assert torch.equal(h[same], h2[same]) and not torch.isfinite(h2[at, c])
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[n, c] = False
        assert torch.equal(out[keep], out2[keep])
        got = backward(e, h)
        same = torch.ones_like(h, dtype=torch.bool)
        same[sum(lens[:n]):at + 1, c] = False
        for m in ("dx", "dg"):
            assert torch.equal(back[m][same], got[m][same]), m
        assert torch.equal(back["dstate_in"][keep], got["dstate_in"][keep])


SEQS = [300, 5, 700, 1, 40, 2100, 64]


def spoilt(d, n, name, value, c, t):
    """d with one element of sequence n changed, and where sequence n's rows are."""
    x = cuda(d)
    at = d["cu"].tolist()
    x[name] = x[name].clone()
    x[name][at[n] + t if t >= 0 else at[n + 1] + t, c] = value
    return x, at[n], at[n + 1]


@pytest.mark.parametrize("n", [0, 2, 3, 5])
@pytest.mark.parametrize("name, value", [("x", float("nan")), ("x", float("inf")), ("g", float("nan")),
                                         ("g", float("inf")), ("state_in", float("nan"))])
@pytest.mark.parametrize("D, gate", [(24, "log"), (23, "logit")])
def test_steep_decays_keep_infinities_in_their_sequence(D, gate, name, value, n):
    """To the end of its sequence, over tiles whose product of decays is 0, and no further, over
    tiles whose product of decays is not a number."""
    if gate == "logit" and name == "g" and value == float("inf"):
        value = float("nan")  # (a logit of infinity is a decay of 1)
    d = ref.make(SEQS, D, gate, False, "f32", "f32", kind="steep", seed=n)
    clean, clean_out = forward(d)
    t = min(3, SEQS[n] - 1)
    if name == "state_in":
        x = cuda(d)
        x["state_in"] = x["state_in"].clone()
        x["state_in"][n, 9] = value
        lo, hi = d["cu"].tolist()[n:n + 2]
        t = 0
    else:
        x, lo, hi = spoilt(d, n, name, value, 9, t)
    h, out = forward(d, x)
    bad = torch.zeros_like(h, dtype=torch.bool)
    bad[lo + t:hi, 9] = True
    assert torch.equal(h[~bad], clean[~bad]) and not torch.isfinite(h[bad]).any()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[n, 9] = True
    assert torch.equal(out[~bad], clean_out[~bad]) and not torch.isfinite(out[bad]).any()


@pytest.mark.parametrize("n", [0, 2, 3, 5])
@pytest.mark.parametrize("name", ["dh", "g"])
@pytest.mark.parametrize("D, gate", [(24, "log"), (23, "logit")])
def test_steep_decays_keep_infinities_in_their_sequence_gradient(D, gate, name, n):
    d = ref.make(SEQS, D, gate, False, "f32", "f32", kind="steep", seed=n)
    h, _ = forward(d)
    clean = backward(d, h)
    t = -min(3, SEQS[n])
    x, lo, hi = spoilt(d, n, name, float("nan"), 9, t)
    got = backward(d, h, x)
    row = hi + t
    # dx_t is r_t, that does not hold a_t; dg_t and dstate_in are a_t r_t
    for out, first in (("dx", row if name == "dh" else row - 1), ("dg", row)):
        bad = torch.zeros_like(got[out], dtype=torch.bool)
        bad[lo:first + 1, 9] = True
        assert torch.equal(got[out][~bad], clean[out][~bad]), out
        assert not torch.isfinite(got[out][bad]).any(), out
    bad = torch.zeros_like(got["dstate_in"], dtype=torch.bool)
    bad[n, 9] = True
    assert torch.equal(got["dstate_in"][~bad], clean["dstate_in"][~bad])
    assert not torch.isfinite(got["dstate_in"][bad]).any()


@pytest.mark.parametrize("gate, complement", FORMS)
@pytest.mark.parametrize("dtype, gdtype", TYPES)
def test_slow_decays_keep_their_precision(gate, complement, dtype, gdtype):
    """States that remember hundreds of tokens, in the 2-norm.  Each step multiplies what it
    keeps by a decay and adds with fp32 roundings, independent from one token to the next:
    sqrt(tokens remembered) of them, 3 of 2^-24 at most, where errors of one sign would give
    as many as tokens."""
    gen = torch.Generator().manual_seed(5)
    lens, D = [1500, 700], 96
    d = ref.make(lens, D, gate, complement, dtype, gdtype, seed=5)
    z = 5 + torch.randn(sum(lens), D, generator=gen, dtype=torch.float64) / 2
    g = z if gate == "logit" else -torch.nn.functional.softplus(-z)
    d["g"] = g.to(ref.DT[gdtype])
    want_h, want_s = ref.forward(d)
    h, out = forward(d)
    keep = float((1 / (1 - ref.terms(d)[0])).mean())
    within = 3 * keep ** 0.5 * 2.0 ** -24
    assert float((out.cpu().double() - want_s).norm() / want_s.norm()) <= within
    got = backward(d, h)
    want, _ = ref.backward(d, h.cpu())
    assert float((got["dstate_in"].cpu().double() - want["dstate_in"]).norm() /
                 want["dstate_in"].norm()) <= within
    if dtype == "f32":
        assert float((h.cpu().double() - want_h).norm() / want_h.norm()) <= within


@pytest.mark.parametrize("N", [62, 63, 64, 65, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_numbers_of_sequences(N, dtype):
    """Short ones, empty ones and a long one, as many as a wave's lanes and about."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 20, (N,), generator=gen).tolist()
    lens[N // 2], lens[-1] = 400, 0
    check_all(ref.make(lens, 40, "logit", True, dtype, "f32", seed=N, pad=5))


@pytest.mark.parametrize("D", [12, 100, 508])
@pytest.mark.parametrize("gdtype", ["bf16", "f32"])
def test_widths_of_four(D, gdtype):
    """fp32 rows of 16-byte loads that bf16's would not have."""
    check_all(ref.make(RAGGED, D, "log", True, "f32", gdtype, seed=D, pad=3))
    check_all(ref.make(RAGGED, D, "log", True, "bf16", gdtype, seed=D, pad=3))


def test_bad_offsets_stay_inside():
    """Offsets that decrease, are negative or pass the end: wrong results, nothing out of range."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make([400], 40, "log", True, "bf16", "bf16", seed=11)
    x = cuda(d)
    guard = torch.full((3 * 400, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 900, 400], [-5, 100, 400], [0, 300, 100, 400], [400, 0], [0, -1, 2 ** 31 - 1],
               [2 ** 31 - 1, -2 ** 31], [50, 60]):
        say(f"channel cu {cu}")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        N = len(cu) - 1
        s = torch.zeros(N, 40, device="cuda")
        h = guard[400:800]
        gdr.gdr_channel_prefill(x["x"], x["g"], c, s, s.clone(), h, **form(d))
        gdr.gdr_channel_backward(x["x"], x["g"], x["dh"], c, s, x["dh"], s, h, x["dh"].clone(),
                                 dstate_in=s.clone(), **form(d))
        torch.cuda.synchronize()
        assert (guard[:400] == 7).all() and (guard[800:] == 7).all()


@pytest.mark.parametrize("N, D", [(1, 1), (3, 77), (64, 4096), (257, 136), (5, 2050)])
@pytest.mark.parametrize("dtype, gdtype", TYPES)
def test_decode(N, D, dtype, gdtype):
    import gated_delta_rule_100_amd as gdr
    for gate, complement in FORMS:
        say(f"channel decode N {N} D {D} {dtype} {gdtype} {gate} {complement}")
        d = ref.make([1] * N, D, gate, complement, dtype, gdtype, seed=N + D)
        x = cuda(d)
        h, state = nan_like(x["x"]), x["state_in"].clone()
        gdr.gdr_channel_decode(x["x"], x["g"], state, h, **form(d))
        torch.cuda.synchronize()
        a, _, b = ref.terms(d)
        s0 = d["state_in"].double()
        want, e = a * s0 + b, ref.step_error(d) * (a * s0.abs() + b.abs())
        ref.check("state", state, want, e)
        ref.check("h", h, want, e)
        # slices of wider rows, h over x
        if D % 8 == 0:
            w = torch.empty(N, 2 * D, dtype=x["x"].dtype, device="cuda")
            w[:, D:] = x["x"]
            s2, h2 = x["state_in"].clone(), nan_like(x["x"])
            gdr.gdr_channel_decode(w[:, D:], x["g"], s2, h2, **form(d))
            gdr.gdr_channel_decode(x["x"], x["g"], x["state_in"], x["x"], **form(d))
            torch.cuda.synchronize()
            assert torch.equal(h, h2) and torch.equal(state, s2)
            assert torch.equal(h, x["x"]) and torch.equal(state, x["state_in"])


def test_tokens_continue_a_prompt():
    import gated_delta_rule_100_amd as gdr
    d = ref.make([40, 55], 64, "logit", True, "f32", "f32", seed=13)
    h, out = forward(d)
    x = cuda(d)
    # sequences cut at 30 and 45
    cu = torch.tensor([0, 30, 75], dtype=torch.int32, device="cuda")
    rows = torch.cat([torch.arange(30), 40 + torch.arange(45)]).cuda()
    s = torch.empty_like(out)
    gdr.gdr_channel_prefill(x["x"][rows], x["g"][rows], cu, x["state_in"], s, h[rows].clone(),
                            **form(d))
    got = []
    for t in range(10):
        at = torch.tensor([30 + t, 40 + 45 + t]).cuda()
        ht = torch.empty(2, 64, device="cuda")
        gdr.gdr_channel_decode(x["x"][at], x["g"][at], s, ht, **form(d))
        got.append((at, ht))
    torch.cuda.synchronize()
    for at, ht in got:
        assert (ht - h[at]).abs().max() < 1e-5
    assert (s - out).abs().max() < 1e-5


def test_repeated_streams_and_graph():
    """Bits do not depend on the order in which workgroups run; a captured call replayed."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make([5000, 70, 0, 3000], 520, "log", True, "bf16", "bf16", kind="slow", seed=14)
    x = cuda(d)
    h, out = forward(d, x)
    want = backward(d, h, x)
    T, D = h.shape
    ws = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
          for n in (gdr.gdr_channel_prefill_workspace_bytes(T, D),
                    gdr.gdr_channel_backward_workspace_bytes(T, D))]
    for w in ws:
        w.random_(0, 256)
    got = [nan_like(h), nan_like(out)] + [nan_like(t) for t in want.values()]

    def step(stream=None):
        gdr.gdr_channel_prefill(x["x"], x["g"], x["cu"], x["state_in"], got[1], got[0], **form(d),
                                workspace=ws[0], stream=stream)
        gdr.gdr_channel_backward(x["x"], x["g"], h, x["cu"], x["state_in"], x["dh"], x["dstate_out"],
                                 got[2], got[3], dstate_in=got[4], workspace=ws[1], stream=stream,
                                 **form(d))

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(got, [h, out, *want.values()]))

    torch.cuda.synchronize()
    for _ in range(5):
        step()
        assert same()
    step(torch.cuda.Stream())
    assert same()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    for r in range(4):
        for t in got:
            t.fill_(float(r))
        torch.cuda.synchronize()
        graph.replay()
        assert same(), r


def test_two_calls_at_once():
    """On two streams with workspaces of their own, given or not."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make([6000], 256, "log", False, "bf16", "bf16", kind="slow", seed=15)
    x = cuda(d)
    h, out = forward(d, x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = [(nan_like(h), nan_like(out)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (a, b) in zip(streams, res):
            gdr.gdr_channel_prefill(x["x"], x["g"], x["cu"], x["state_in"], b, a, stream=s, **form(d))
    torch.cuda.synchronize()
    for a, b in res:
        assert torch.equal(a, h) and torch.equal(b, out)


@pytest.mark.parametrize("D", [2048, 2050])
def test_more_than_2_31_elements(D):
    import gated_delta_rule_100_amd as gdr
    L, T = 300, (1 << 31) // 2048 + 700
    say(f"channel T {T} D {D}")
    d = ref.make([L], D, "log", True, "bf16", "bf16", seed=16)
    x, g = (torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-L:], g[-L:] = d["x"].cuda(), d["g"].cuda()
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device="cuda")
    s = torch.zeros(2, D, device="cuda")
    s[1] = d["state_in"][0].cuda()
    out, h = torch.empty_like(s), torch.empty_like(x)
    gdr.gdr_channel_prefill(x, g, cu, s, out, h, **form(d))
    torch.cuda.synchronize()
    want_h, want_s = ref.forward(d)
    eh, es = ref.forward_bounds(d)
    ref.check("h", h[-L:], want_h, eh)
    ref.check("state_out", out[1:], want_s, es)
    assert not h[:-L].any()
    dh = torch.zeros_like(x)
    dh[-L:] = d["dh"].cuda()
    want, bounds = ref.backward(d, h[-L:].cpu())
    ds, dsi = torch.zeros_like(s), torch.empty_like(s)
    ds[1] = d["dstate_out"][0].cuda()
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    gdr.gdr_channel_backward(x, g, h, cu, s, dh, ds, dx, dg, dstate_in=dsi, **form(d))
    torch.cuda.synchronize()
    for n, t in (("dx", dx[-L:]), ("dg", dg[-L:]), ("dstate_in", dsi[1:])):
        ref.check(n, t, want[n], bounds[n])
    assert not dx[:-L].any() and not dg[:-L].any() and not dsi[0].any()
