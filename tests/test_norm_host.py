"""Norms around a block: refusals of the entry points before a device is touched, and the
reference's gradients against central differences."""
import ctypes
import os

import pytest
import torch

import norm_ref as ref

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    import gated_delta_rule_100_amd as g
    if not os.path.exists(g.library_path()):
        from gated_delta_rule_100_amd.build import build_library
        build_library()
    return g._load()


def test_reference_gradients_against_differences():
    for kw in (dict(), dict(gate="sigmoid", residual=False), dict(after=False, before=False)):
        d = ref.make(3, 5, "f32", seed=4, **kw)
        grads = ref.backward(d)
        gen = torch.Generator().manual_seed(1)
        for name in [n[1:] for n in grads]:
            base = {n: d[n].double() for n in ("x", "w_after", "gate", "residual", "w_before")
                    if d[n] is not None}
            step = torch.randn(base[name].shape, generator=gen, dtype=torch.float64)

            def loss(s):
                h, y = ref.forward(d, dict(base, **{name: base[name] + s * step}))
                out = (h * d["dh"].double()).sum()
                return float(out if y is None else out + (y * d["dy"].double()).sum())

            eps = 1e-6
            want = float((grads["d" + name] * step).sum())
            assert abs((loss(eps) - loss(-eps)) / (2 * eps) - want) < 1e-6 * max(1, abs(want)), name


def _forward(lib, **over):
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    a = dict(x=FAKE, wa=FAKE, z=FAKE, r=FAKE, wb=FAKE, h=FAKE + 64, y=FAKE + 128, rows=4, D=64,
             scale=1.0, eps=1e-6, act=0, ind=0, wd=0, outd=0)
    a.update(over)
    return lib.gdr_block_norm(p(a["x"]), p(a["wa"]), p(a["z"]), p(a["r"]), p(a["wb"]), p(a["h"]),
                              p(a["y"]), a["rows"], a["D"], a["scale"], a["eps"], a["act"],
                              a["ind"], a["wd"], a["outd"], None)


def _backward(lib, **over):
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    a = dict(x=FAKE, wa=FAKE, z=FAKE, r=FAKE, wb=FAKE, dh=FAKE, dy=FAKE, dx=FAKE, dz=FAKE, dr=FAKE,
             dwa=FAKE, dwb=FAKE, rows=4, D=64, scale=1.0, eps=1e-6, act=0, ind=0, wd=0, outd=0,
             ws=FAKE, wsb=1 << 30)
    a.update(over)
    return lib.gdr_block_norm_backward(
        *(p(a[n]) for n in ("x", "wa", "z", "r", "wb", "dh", "dy", "dx", "dz", "dr", "dwa", "dwb")),
        a["rows"], a["D"], a["scale"], a["eps"], a["act"], a["ind"], a["wd"], a["outd"],
        p(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("call", [_forward, _backward])
@pytest.mark.parametrize("over, status, word", [
    (dict(x=None), 1, "NULL"), (dict(rows=-1), 1, "rows"), (dict(rows=1 << 31), 1, "rows"),
    (dict(rows=(1 << 28) + 1, D=1), 1, "rows"), (dict(rows=1 << 20, D=8192), 1, "rows"),
    (dict(D=0), 2, "D=0"), (dict(D=16385), 2, "D=16385"), (dict(act=2), 1, "act"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(ind=2), 2, "dtype"),
    (dict(wd=3), 2, "dtype"), (dict(outd=-1), 2, "dtype"), (dict(r=FAKE + 4), 1, "aligned"),
])
def test_refusals(lib, call, over, status, word):
    assert call(lib, **over) == status
    assert word in lib.gdr_last_error().decode()


def test_more_refusals(lib):
    for over, word in ((dict(y=None), "exactly"), (dict(wb=None), "exactly"),
                       (dict(h=None, y=None), "NULL"), (dict(y=FAKE + 64), "one buffer"),
                       (dict(h=FAKE, outd=1), "in place")):
        assert _forward(lib, **over) == 1
        assert word in lib.gdr_last_error().decode()
    for over, word in ((dict(dy=None), "exactly"), (dict(wb=None, dwb=None), "exactly"),
                       (dict(dx=None), "NULL"), (dict(dh=None, dy=None), "NULL"),
                       (dict(z=None), "not given"), (dict(wa=None), "not given"),
                       (dict(wsb=16), "workspace"), (dict(ws=None), "workspace"),
                       (dict(ws=FAKE + 8), "aligned")):
        assert _backward(lib, **over) == 1
        assert word in lib.gdr_last_error().decode()


def test_workspace_sizes(lib):
    import gated_delta_rule_100_amd as g
    assert g.gdr_block_norm_backward_workspace_bytes(-1, 64) == 0
    assert g.gdr_block_norm_backward_workspace_bytes(10, 16385) == 0
    assert g.gdr_block_norm_backward_workspace_bytes(0, 64) == 0
    assert g.gdr_block_norm_backward_workspace_bytes(10000, 2048) >= 2 * 4 * 2048


def test_binding_refuses(lib):
    import gated_delta_rule_100_amd as g
    x = torch.zeros(2, 8)
    with pytest.raises(g.GdrError, match="GPU"):
        g.gdr_block_norm(x, x)
    with pytest.raises(g.GdrError, match="row operands"):
        g.gdr_block_norm(x, x, gate=x.bfloat16())
    with pytest.raises(g.GdrError, match="weights"):
        g.gdr_block_norm(x, x, w_after=torch.zeros(4))
    with pytest.raises(g.GdrError, match="outputs"):
        g.gdr_block_norm(x, x, torch.zeros(2, 4), w_before=torch.zeros(8))
    with pytest.raises(g.GdrError, match="act"):
        g.gdr_block_norm(x, x, gate=x, act="gelu")
    with pytest.raises(g.GdrError, match="weight gradients"):
        g.gdr_block_norm_backward(x, x, None, x, w_after=torch.zeros(8), dw_after=torch.zeros(4))
