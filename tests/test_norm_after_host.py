"""norm= of the recurrences without a GPU: the library is the real one where a call validates on
the host, tensors are without memory, and launches are recorded."""
import os

import pytest
import torch

RECURRENCES = ("gdr_decode_step", "gdr_decode_mtp", "gdr_chunk_prefill",
               "gdr_chunk_prefill_noalloc", "gdr_linear_decode", "gdr_linear_prefill")


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def call(g, name, tokens, H, norm, d=128, **kw):
    """One call of a recurrence with `tokens` tokens (in decode: sequences) and its norm."""
    f32 = torch.float32
    gates, o = meta(tokens, H, dtype=f32), meta(tokens, H, d)
    q = meta(tokens, H, d)
    cu, state = meta(2, dtype=torch.int32), meta(1, H, d, d, dtype=f32)
    norm = dict(norm, h=meta(*o.shape))
    if name == "gdr_decode_step":
        return g.gdr_decode_step(q, q, q, gates, gates, meta(tokens, H, d, d, dtype=f32), o,
                                 norm=norm, **kw)
    if name == "gdr_decode_mtp":
        norm["h"] = norm["h"][:, None]
        return g.gdr_decode_mtp(q[:, None], q[:, None], q[:, None], gates[:, None], gates[:, None],
                                meta(tokens, H, d, d, dtype=f32), None, o[:, None], norm=norm, **kw)
    if name.startswith("gdr_chunk"):
        return getattr(g, name)(q, q, q, gates, gates, cu, None, state, o, norm=norm, **kw)
    if name == "gdr_linear_decode":
        return g.gdr_linear_decode(q, q, q, gates, meta(tokens, H, d, d, dtype=f32), o, norm=norm,
                                   **kw)
    return g.gdr_linear_prefill(q, q, q, gates, cu, None, state, o, norm=norm, **kw)


class Recorder:
    """Stands for the library: entries that launch are recorded as (name, device, stream), the
    others go to the real library."""

    def __init__(self, lib, current):
        self._lib, self._current, self.launches = lib, current, []

    def __getattr__(self, name):
        real = getattr(self._lib, name)
        if name not in RECURRENCES + ("gdr_block_norm",):
            return real

        def entry(*args):
            if name == "gdr_block_norm" and args[7] == 0:
                return real(*args)
            self.launches.append((name, self._current[-1], args[-1]))
            return 0
        return entry


@pytest.fixture
def host(monkeypatch):
    """The package on a machine that claims two GPUs, 0 the current one; tensors are on `home`,
    whose current stream is 100 + home."""
    import gated_delta_rule_100_amd as g
    if not os.path.exists(g.library_path()):
        from gated_delta_rule_100_amd.build import build_library
        build_library()
    current, home = [0], [0]

    class On:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            current.append(self.dev)

        def __exit__(self, *a):
            current.pop()

    class Stream:
        @property
        def cuda_stream(self):
            return 100 + current[-1]

    lib = Recorder(g._load(), current)
    monkeypatch.setattr(g, "_lib", lib)
    monkeypatch.setattr(g, "_device", lambda t, name: home[0])
    monkeypatch.setattr(g, "_ptr", lambda t, name, dtypes, dev: None if t is None else 0x10000)
    monkeypatch.setattr(g, "_dev_ptr", lambda t, name, dtypes=None, optional=False:
                        None if t is None else 0x10000)
    monkeypatch.setattr(g, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream())
    monkeypatch.setattr(torch.cuda, "device", On)
    return g, lib, home


@pytest.mark.parametrize("name", RECURRENCES)
def test_rows_that_the_norm_refuses_are_refused_before_anything_runs(host, name):
    g, lib, _ = host
    ws = dict(workspace=meta(1, dtype=torch.uint8)) if name in ("gdr_chunk_prefill",
                                                                "gdr_linear_prefill") else {}
    # rows * D = 2^33 at 128 values a row
    with pytest.raises(g.GdrError, match="rows=67108864"):
        call(g, name, 1 << 16, 1 << 10, {}, **ws)
    assert lib.launches == []
    call(g, name, 1 << 10, 16, {}, **ws)
    assert [n for n, _, _ in lib.launches] == [name, "gdr_block_norm"]


@pytest.mark.parametrize("name", RECURRENCES)
@pytest.mark.parametrize("stream", [None, 7])
def test_the_norm_follows_its_recurrence_on_the_stream_of_their_device(host, name, stream):
    """With everything on GPU 1 while GPU 0 is the current one."""
    g, lib, home = host
    home[0] = 1
    ws = dict(workspace=meta(1, dtype=torch.uint8)) if name in ("gdr_chunk_prefill",
                                                                "gdr_linear_prefill") else {}
    call(g, name, 128, 4, {}, stream=stream, **ws)
    on = 101 if stream is None else stream
    assert lib.launches == [(name, 1, on), ("gdr_block_norm", 1, on)]
