"""The recurrence with a decay for each channel without a GPU: the reference's gradient formulas
against autograd and differences, and refusals before a device is touched."""
import ctypes
import os

import pytest
import torch

import channel_ref as ref

FAKE = 0x10000  # never dereferenced: validation fails first
FORMS = [("log", False), ("log", True), ("logit", False), ("logit", True)]


@pytest.fixture(scope="module")
def lib():
    import gated_delta_rule_100_amd as g
    if not os.path.exists(g.library_path()):
        from gated_delta_rule_100_amd.build import build_library
        build_library()
    return g._load()


@pytest.mark.parametrize("gate, complement", FORMS)
def test_reference_gradients(gate, complement):
    d = ref.make([5, 0, 1, 9], 3, gate, complement, "f32", seed=3)
    h, _ = ref.forward(d)
    want, _ = ref.backward(d, h)
    auto = ref.autograd(d)
    for n in want:
        assert (want[n] - auto[n]).abs().max() < 1e-12, n
    # and a difference along a random direction
    gen = torch.Generator().manual_seed(1)
    leaves = {n: d[n].to(ref.F64) for n in ("x", "g", "state_in")}
    step = {n: torch.randn(t.shape, generator=gen, dtype=ref.F64) for n, t in leaves.items()}

    def loss(s):
        h, end = ref.forward(d, {n: t + s * step[n] for n, t in leaves.items()})
        return float((h * d["dh"].to(ref.F64)).sum() + (end * d["dstate_out"].to(ref.F64)).sum())

    got = sum(float((want["d" + n] * step[n]).sum()) for n in leaves)
    assert abs((loss(1e-6) - loss(-1e-6)) / 2e-6 - got) < 1e-6 * max(1, abs(got))


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x)


def _decode(lib, **over):
    a = dict(x=FAKE, g=FAKE, s=FAKE, h=FAKE, N=2, D=64, xs=0, gs=0, gate=0, comp=0, io=0, gd=0)
    a.update(over)
    return lib.gdr_channel_decode(*(_ptr(a[n]) for n in ("x", "g", "s", "h")), a["N"], a["D"],
                                  a["xs"], a["gs"], a["gate"], a["comp"], a["io"], a["gd"], None)


def _prefill(lib, **over):
    a = dict(x=FAKE, g=FAKE, cu=FAKE, N=2, si=None, so=FAKE, h=FAKE, T=300, D=64, xs=0, gs=0,
             gate=0, comp=0, io=0, gd=0, ws=FAKE, wsb=1 << 40)
    a.update(over)
    return lib.gdr_channel_prefill(_ptr(a["x"]), _ptr(a["g"]), _ptr(a["cu"]), a["N"], _ptr(a["si"]),
                                   _ptr(a["so"]), _ptr(a["h"]), a["T"], a["D"], a["xs"], a["gs"],
                                   a["gate"], a["comp"], a["io"], a["gd"], _ptr(a["ws"]), a["wsb"],
                                   None)


def _backward(lib, **over):
    a = dict(x=FAKE, g=FAKE, h=FAKE, cu=FAKE, N=2, si=None, dh=FAKE, dso=None, dx=FAKE, dg=FAKE,
             dsi=None, T=300, D=64, xs=0, gs=0, gate=0, comp=0, io=0, gd=0, ws=FAKE, wsb=1 << 40)
    a.update(over)
    return lib.gdr_channel_backward(_ptr(a["x"]), _ptr(a["g"]), _ptr(a["h"]), _ptr(a["cu"]), a["N"],
                                    *(_ptr(a[n]) for n in ("si", "dh", "dso", "dx", "dg", "dsi")),
                                    a["T"], a["D"], a["xs"], a["gs"], a["gate"], a["comp"],
                                    a["io"], a["gd"], _ptr(a["ws"]), a["wsb"], None)


BAD = [(dict(D=0), 2), (dict(D=(1 << 20) + 1), 2), (dict(N=0), 1), (dict(N=(1 << 20) + 1), 1),
       (dict(N=1 << 20, D=1 << 11), 1), (dict(xs=63), 1), (dict(gs=(1 << 24) + 1), 1),
       (dict(gate=2), 1), (dict(comp=2), 1), (dict(io=2), 2), (dict(gd=-1), 2), (dict(g=FAKE + 8), 1),
       (dict(g=None), 1), (dict(h=None), 1)]


@pytest.mark.parametrize("over, status", BAD)
def test_refusals(lib, over, status):
    for call in (_decode, _prefill, _backward):
        assert call(lib, **over) == status, (call.__name__, over)
        assert lib.gdr_last_error().decode().startswith("gdr_channel" + call.__name__)


def test_refusals_of_one_entry(lib):
    assert _decode(lib, x=None) == _decode(lib, s=None) == 1
    assert _decode(lib, xs=128) == 1  # in place needs a dense x
    assert _prefill(lib, x=None) == _prefill(lib, cu=None) == _prefill(lib, T=-1) == 1
    assert _prefill(lib, xs=128) == 1
    assert _prefill(lib, T=1 << 30, D=1 << 14) == 1
    assert "more than a launch holds" in lib.gdr_last_error().decode()
    assert _prefill(lib, so=FAKE + 4) == _prefill(lib, si=FAKE + 4) == 1
    for n in ("dh", "dx", "dg", "cu"):
        assert _backward(lib, **{n: None}) == 1, n
    assert _backward(lib, x=None, comp=1) == 1
    for n in ("dh", "dx", "dg", "dso", "dsi", "si"):
        assert _backward(lib, **{n: FAKE + 4}) == 1, n


@pytest.mark.parametrize("T, D", [(0, 64), (64, 100), (300, 64), (16384, 2048), (131072, 512)])
def test_workspace(lib, T, D):
    import gated_delta_rule_100_amd as g
    for call, size in ((_prefill, g.gdr_channel_prefill_workspace_bytes),
                       (_backward, g.gdr_channel_backward_workspace_bytes)):
        need = size(T, D)
        assert need <= 64 + T * D  # far below a tensor of the pass
        if need:
            assert call(lib, T=T, D=D, wsb=need - 1) == 1
            assert "workspace" in lib.gdr_last_error().decode()
            assert call(lib, T=T, D=D, ws=None) == 1
            assert call(lib, T=T, D=D, ws=FAKE + 8) == 1
        assert size(-1, D) == size(T, 0) == size(1 << 30, 1 << 20) == 0


def test_binding_refuses(lib):
    import gated_delta_rule_100_amd as g
    x = torch.zeros(4, 8)
    cu = torch.zeros(2, dtype=torch.int32)
    s = torch.zeros(1, 8)
    with pytest.raises(g.GdrError, match="on the GPU"):
        g.gdr_channel_prefill(x, x, cu, None, None, x)
    with pytest.raises(g.GdrError, match="on the GPU"):
        g.gdr_channel_backward(x, x, x, cu, None, x, None, x, x)
    with pytest.raises(g.GdrError, match="on the GPU"):
        g.gdr_channel_decode(x, x, x.clone(), x)
    with pytest.raises(g.GdrError, match="gate must be"):
        g.gdr_channel_decode(x, x, x.clone(), x, gate="tanh")
    with pytest.raises(g.GdrError, match="share a dtype"):
        g.gdr_channel_prefill(x, x, cu, None, None, x.bfloat16())
    with pytest.raises(g.GdrError, match="state_in must have shape"):
        g.gdr_channel_prefill(x, x, cu, torch.zeros(2, 8), None, x)
    with pytest.raises(g.GdrError, match="inconsistent shapes"):
        g.gdr_channel_backward(x, x, x, cu, None, x, None, x, s)
