"""Linear attention with a decay for each head, checks that need no GPU: the
reference of the GPU tests against the token-by-token recurrence and central
differences, and every refusal of the entry points before a device is touched."""
import ctypes
import os

import pytest
import torch

import linear_ref as ref

CASES = [
    dict(lens=[5, 0, 70, 1], H=4, Hk=2, dk=64, dv=128, decay="token", gate="std"),
    dict(lens=[33, 2], H=2, Hk=2, dk=64, dv=64, decay="head", gate="slow"),
    dict(lens=[40], H=2, Hk=1, dk=128, dv=64, decay="token", gate="reset", state=False),
]


def _recurrence(d):
    x = ref.inputs64(d)
    H = d["H"]
    rep = lambda t: t.repeat_interleave(H // t.shape[1], 1)  # noqa: E731
    q, k, v = rep(x["q"]), rep(x["k"]), x["v"]
    g = x["g"] if x["g"].dim() == 2 else x["g"].expand(q.shape[0], H)
    o, out = torch.zeros_like(v), []
    for n, L in enumerate(d["lens"]):
        S = x["state_in"][n].clone() if x["state_in"] is not None else \
            torch.zeros(H, d["dv"], d["dk"], dtype=torch.float64)
        for t in range(int(d["cu"][n]), int(d["cu"][n]) + L):
            S = g[t].exp()[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = d["scale"] * (S @ q[t][:, :, None])[..., 0]
        out.append(S)
    return o, torch.stack(out)


@pytest.mark.parametrize("case", CASES)
def test_reference_is_the_recurrence(case):
    d = ref.make(seed=3, dtype="f32", **case)
    o, s = ref.forward(d)
    o2, s2 = _recurrence(d)
    assert (o - o2).abs().max() < 1e-12 * (1 + o2.abs().max())
    assert (s - s2).abs().max() < 1e-12 * (1 + s2.abs().max())


def test_reference_gradients_against_differences():
    d = ref.make([7, 3], 2, 1, 64, 64, dtype="f32", decay="token", gate="std", seed=5)
    grads = ref.backward(d)
    gen = torch.Generator().manual_seed(1)
    eps = 1e-6

    def loss(x):
        o, s = ref.forward(d, leaves=x)
        return float((o * x["do"]).sum() + (s * x["dstate_out"]).sum())

    for name in ("q", "k", "v", "g", "state_in"):
        x = ref.inputs64(d)
        step = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        base = x[name].clone()
        x[name] = base + eps * step
        hi = loss(x)
        x[name] = base - eps * step
        lo = loss(x)
        want = float((grads["d" + name] * step).sum())
        # truncation eps^2 f''' and cancellation 2^-53 |loss| / eps, both below 1e-6 of the value
        assert abs((hi - lo) / (2 * eps) - want) < 1e-5 * max(1.0, abs(want)), name


@pytest.fixture(scope="module")
def lib():
    import gated_delta_rule_100_amd as g
    if not os.path.exists(g.library_path()):
        from gated_delta_rule_100_amd.build import build_library
        build_library()
    return g._load()


FAKE = 0x10000  # never dereferenced: validation fails first


def _call(lib, entry, over):
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=FAKE, N=2, sin=None, sout=FAKE, o=FAKE, do=FAKE,
             dso=None, dq=FAKE, dkk=FAKE, dvv=FAKE, dg=None, dsi=None, T=100, H=4, Hk=2, dk=128,
             dv=64, qs=0, ks=0, vs=0, scale=1.0, decay=0, ind=0, outd=0, ws=None, wsb=0, state=FAKE)
    a.update(over)
    tail = [a["H"], a["Hk"], a["dk"], a["dv"], a["qs"], a["ks"], a["vs"], a["scale"], a["decay"],
            a["ind"], a["outd"]]
    if entry == "decode":
        return lib.gdr_linear_decode(p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), p(a["state"]),
                                     p(a["o"]), a["N"], *tail, None)
    if entry == "prefill":
        return lib.gdr_linear_prefill(p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), p(a["cu"]),
                                      a["N"], p(a["sin"]), p(a["sout"]), p(a["o"]), a["T"], *tail,
                                      p(a["ws"]), a["wsb"], None)
    return lib.gdr_linear_backward(p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), p(a["cu"]), a["N"],
                                   p(a["sin"]), p(a["do"]), p(a["dso"]), p(a["dq"]), p(a["dkk"]),
                                   p(a["dvv"]), p(a["dg"]), p(a["dsi"]), a["T"], *tail,
                                   p(a["ws"]), a["wsb"], None)


SHARED = [
    (dict(q=None), 1, "NULL"), (dict(v=None), 1, "NULL"), (dict(g=None), 1, "NULL"),
    (dict(N=0), 1, "N=0"), (dict(H=0), 1, "H=0"), (dict(Hk=0), 1, "Hk=0"),
    (dict(H=5), 1, "multiple"), (dict(dk=96), 2, "(96, 64)"), (dict(dv=256), 2, "(128, 256)"),
    (dict(ind=2), 2, "dtype"), (dict(outd=-1), 2, "dtype"), (dict(decay=2), 1, "decay"),
    (dict(qs=255), 1, "q_stride"), (dict(qs=260), 1, "q_stride"), (dict(ks=-256), 1, "k_stride"),
    (dict(vs=128), 1, "v_stride"), (dict(ks=(1 << 24) + 8), 1, "2^24"),
    (dict(N=1 << 15, H=128), 1, "large"), (dict(N=70000), 1, "large"), (dict(k=FAKE + 8), 1, "aligned"),
]


@pytest.mark.parametrize("entry", ["decode", "prefill", "backward"])
@pytest.mark.parametrize("over, status, word", SHARED)
def test_refusals(lib, entry, over, status, word):
    assert _call(lib, entry, over) == status
    assert word in lib.gdr_last_error().decode()
    assert "gdr_linear_" + entry in lib.gdr_last_error().decode()


@pytest.mark.parametrize("entry, over, status, word", [
    ("decode", dict(state=None), 1, "NULL"),
    ("decode", dict(o=FAKE + 4), 1, "aligned"),
    ("prefill", dict(cu=None), 1, "NULL"),
    ("prefill", dict(o=None), 1, "NULL"),
    ("prefill", dict(T=-1), 1, "tokens=-1"),
    ("prefill", dict(T=1 << 30, H=4), 1, "large"),
    ("prefill", dict(N=1, T=1 << 20, wsb=1), 1, "workspace"),
    ("backward", dict(do=None), 1, "NULL"),
    ("backward", dict(dq=None), 1, "NULL"),
    ("backward", dict(dsi=FAKE, dso=FAKE), 1, "dstate_in"),
    ("backward", dict(wsb=64), 1, "workspace"),
])
def test_more_refusals(lib, entry, over, status, word):
    if entry == "prefill" and word == "workspace" and \
            lib.gdr_linear_prefill_workspace_bytes(over["T"], 1, 4, 128, 64, 0) == 0:
        pytest.skip("this call needs no workspace")
    assert _call(lib, entry, over) == status
    assert word in lib.gdr_last_error().decode()


def test_workspace_sizes(lib):
    import gated_delta_rule_100_amd as g
    for bad in ((-1, 1, 4, 2, 64, 64), (10, 0, 4, 2, 64, 64), (10, 1, 4, 3, 64, 64),
                (10, 1, 4, 2, 96, 64)):
        assert g.gdr_linear_backward_workspace_bytes(*bad) == 0
    assert g.gdr_linear_prefill_workspace_bytes(100, 1, 4, 96, 64) == 0
    # shared heads add the value heads' own dq and dk in fp32
    own = g.gdr_linear_backward_workspace_bytes(100, 2, 4, 4, 64, 64, torch.float32)
    shared = g.gdr_linear_backward_workspace_bytes(100, 2, 4, 2, 64, 64, torch.float32)
    assert own > 0 and shared >= own + 2 * 100 * 4 * 64 * 4


def test_binding_refuses(lib):
    import gated_delta_rule_100_amd as g
    q = torch.zeros(2, 2, 64)
    cu = torch.tensor([0, 2], dtype=torch.int32)
    s = torch.zeros(2, 2, 64, 64)
    with pytest.raises(g.GdrError, match="GPU"):
        g.gdr_linear_decode(q, q, q, torch.zeros(2, 2), s, q)
    with pytest.raises(g.GdrError, match="shapes"):
        g.gdr_linear_decode(q, q[:1], q, torch.zeros(2, 2), s, q)
    with pytest.raises(g.GdrError, match="share a dtype"):
        g.gdr_linear_prefill(q, q.bfloat16(), q, torch.zeros(2, 2), cu, None, None, q)
    with pytest.raises(g.GdrError, match="state_in"):
        g.gdr_linear_prefill(q, q, q, torch.zeros(2, 2), cu, s, None, q)
    with pytest.raises(g.GdrError, match="shapes"):
        g.gdr_linear_backward(q, q, q, torch.zeros(2), cu, None, q, None, q, q, q,
                              dg=torch.zeros(3))
