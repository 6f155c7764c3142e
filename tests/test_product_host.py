"""The product in 8 bits and the norm in 8 bits without a GPU: the reference, and refusals before
a device is touched, those of norm= of the recurrences among them."""
import ctypes

import pytest
import torch

import product_ref as ref
from test_norm_after_host import RECURRENCES, host, meta  # noqa: F401

FAKE = 0x10000  # never dereferenced: validation fails first
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    import os

    import gated_delta_rule_100_amd as g
    if not os.path.exists(g.library_path()):
        from gated_delta_rule_100_amd.build import build_library
        build_library()
    return g._load()


def test_reference_against_the_formula():
    d = ref.make(5, 131, 272, seed=1)
    want = torch.zeros(5, 131, dtype=torch.float64)
    for m in range(5):
        for n in range(131):
            for b in range(3):
                k = slice(128 * b, min(272, 128 * b + 128))
                want[m, n] += (d["a"][m, k].double() * d["w"][n, k].double()).sum() * \
                    d["sa"][m, b].double() * d["sw"][n // 128, b].double()
    assert (ref.product(d)[0] - want).abs().max() <= 1e-12 * want.abs().max()


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x)


def _product(lib, **over):
    a = dict(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, out=FAKE, M=4, N=4, K=64, outd=0)
    a.update(over)
    return lib.gdr_product8(*(_ptr(a[n]) for n in ("a", "sa", "w", "sw", "out")), a["M"], a["N"],
                            a["K"], a["outd"], None)


def test_product_refusals(lib):
    for n in ("a", "sa", "w", "sw", "out"):
        assert _product(lib, **{n: None}) == 1, n
        assert _product(lib, **{n: FAKE + 8}) == 1, n
    for over in (dict(M=-1), dict(N=0), dict(K=0), dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 1),
                 dict(M=1 << 24, N=1 << 24)):
        assert _product(lib, **over) == 1, over
    for over in (dict(K=8), dict(K=100), dict(outd=2), dict(outd=-1)):
        assert _product(lib, **over) == 2, over
    assert _product(lib, M=0) == 0  # nothing to do, before a device is looked for


def _norm8(lib, **over):
    a = dict(x=FAKE, wa=FAKE, z=FAKE, r=FAKE, wb=FAKE, h=FAKE + 64, y8=FAKE + 128, ys=FAKE + 192,
             rows=4, D=64, scale=1.0, eps=1e-6, act=0, ind=0, wd=0, outd=0)
    a.update(over)
    return lib.gdr_block_norm8(*(_ptr(a[n]) for n in ("x", "wa", "z", "r", "wb", "h", "y8", "ys")),
                               a["rows"], a["D"], a["scale"], a["eps"], a["act"], a["ind"], a["wd"],
                               a["outd"], None)


def test_norm8_refusals(lib):
    for n in ("x", "y8", "ys"):
        assert _norm8(lib, **{n: None}) == 1, n
    for n in ("x", "wa", "z", "r", "wb", "h", "y8", "ys"):
        assert _norm8(lib, **{n: FAKE + 8}) == 1, n
    for over in (dict(rows=-1), dict(rows=(1 << 28) + 1), dict(eps=-1.0), dict(act=2),
                 dict(y8=FAKE), dict(y8=FAKE + 192), dict(h=FAKE, outd=1)):
        assert _norm8(lib, **over) == 1, over
    for over in (dict(D=0), dict(D=24), dict(D=16400), dict(ind=2), dict(wd=2), dict(outd=2)):
        assert _norm8(lib, **over) == 2, over
    assert _norm8(lib, rows=0, x=None) == 0


def test_binding_refuses(lib):
    import gated_delta_rule_100_amd as g
    x = torch.zeros(4, 256)
    s = torch.zeros(4, 2)
    with pytest.raises(g.GdrError, match="on the GPU"):
        g.gdr_product8(x.to(E4M3), s, x.to(E4M3), s[:1], torch.zeros(4, 4))
    with pytest.raises(g.GdrError, match="inconsistent shapes"):
        g.gdr_product8(x.to(E4M3), s, x.to(E4M3), s, torch.zeros(4, 4))
    with pytest.raises(g.GdrError, match="on the GPU"):
        g.gdr_block_norm8(x, x.to(E4M3), s)


# ---------------------------------------------------------------- behind a recurrence

def norm8(tokens, H, d=128, rows=None, **kw):
    F = 96
    K = rows or H * d
    return dict(h=None, y8=meta(tokens, H, d, dtype=E4M3),
                y_scale=meta(tokens, H, 1, dtype=torch.float32),
                project=dict(w=meta(F, K, dtype=E4M3), out=meta(tokens, F),
                             w_scale=meta(1, -(-K // 128), dtype=torch.float32)), **kw)


@pytest.fixture
def host8(host, monkeypatch):  # noqa: F811
    """host with the 8-bit entries recorded too."""
    g, lib, home = host
    real = type(lib).__getattr__

    def entry(self, name):
        if name not in ("gdr_block_norm8", "gdr_product8"):
            return real(self, name)

        def run(*args):
            if args[8 if name == "gdr_block_norm8" else 5] == 0:  # no rows: the library's checks
                return getattr(self._lib, name)(*args)
            self.launches.append((name, self._current[-1], args[-1]))
            return 0
        return run

    monkeypatch.setattr(type(lib), "__getattr__", entry)
    at = {}  # an address for each argument
    monkeypatch.setattr(g, "_ptr", lambda t, name, dtypes, dev: None if t is None else
                        at.setdefault(name, 0x10000 + 64 * len(at)))
    return g, lib, home


def run_after(g, name, tokens, H, norm, **kw):
    """One call of a recurrence with `tokens` tokens (in decode: sequences) and what follows it."""
    f32, norm = torch.float32, dict(norm)
    gates, o, q = meta(tokens, H, dtype=f32), meta(tokens, H, 128), meta(tokens, H, 128)
    cu, state = meta(2, dtype=torch.int32), meta(1, H, 128, 128, dtype=f32)
    states = meta(tokens, H, 128, 128, dtype=f32)
    if name == "gdr_decode_step":
        return g.gdr_decode_step(q, q, q, gates, gates, states, o, norm=norm, **kw)
    if name == "gdr_decode_mtp":
        norm.update(y8=norm["y8"][:, None], y_scale=norm["y_scale"][:, None],
                    project=dict(norm["project"], out=norm["project"]["out"][:, None]))
        if norm.get("gate") is not None:
            norm["gate"] = norm["gate"][:, None]
        return g.gdr_decode_mtp(q[:, None], q[:, None], q[:, None], gates[:, None], gates[:, None],
                                states, None, o[:, None], norm=norm, **kw)
    if name.startswith("gdr_chunk"):
        return getattr(g, name)(q, q, q, gates, gates, cu, None, state, o, norm=norm, **kw)
    if name == "gdr_linear_decode":
        return g.gdr_linear_decode(q, q, q, gates, states, o, norm=norm, **kw)
    return g.gdr_linear_prefill(q, q, q, gates, cu, None, state, o, norm=norm, **kw)


def workspace(name):
    return dict(workspace=meta(1, dtype=torch.uint8)) if name in ("gdr_chunk_prefill",
                                                                  "gdr_linear_prefill") else {}


@pytest.mark.parametrize("name", RECURRENCES)
@pytest.mark.parametrize("stream", [None, 7])
def test_norm_and_product_follow_on_the_stream_of_their_device(host8, name, stream):
    g, lib, home = host8
    home[0] = 1
    run_after(g, name, 128, 4, norm8(128, 4), stream=stream, **workspace(name))
    on = 101 if stream is None else stream
    assert lib.launches == [(n, 1, on) for n in (name, "gdr_block_norm8", "gdr_product8")]


@pytest.mark.parametrize("name", RECURRENCES)
def test_nothing_runs_where_what_follows_is_refused(host8, name):
    g, lib, _ = host8
    ws = workspace(name)
    for bad, match in ((norm8(128, 4, rows=384), "rows of w"), (norm8(128, 4, eps=-1.0), "eps"),
                       (dict(norm8(128, 4), act="tanh", gate=meta(128, 4, 128)),
                        "act must be")):
        with pytest.raises(g.GdrError, match=match):
            run_after(g, name, 128, 4, bad, **ws)
    wrong = norm8(128, 4)
    wrong["project"]["out"] = meta(128, 95)
    with pytest.raises(g.GdrError, match="out must have shape"):
        run_after(g, name, 128, 4, wrong, **ws)
    wrong = norm8(128, 4)
    wrong["project"]["w_scale"] = meta(1, 3, dtype=torch.float32)
    with pytest.raises(g.GdrError, match="inconsistent shapes"):
        run_after(g, name, 128, 4, wrong, **ws)
    assert lib.launches == []
