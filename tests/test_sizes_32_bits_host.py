"""Sizes past 32 bits without a GPU: the library's are of 32 bits, and the binding refuses others
instead of passing on what is left of them (fixtures with recorded launches)."""
import pytest
import torch

from test_norm_after_host import host, meta  # noqa: F401
from test_product_host import E4M3, host8  # noqa: F401

F32, MORE = torch.float32, (1 << 32) + 5


@pytest.fixture
def all_recorded(host8, monkeypatch):  # noqa: F811
    g, lib, _ = host8
    real = type(lib).__getattr__

    def entry(self, name):
        if name in ("gdr_channel_decode", "gdr_channel_prefill", "gdr_channel_backward"):
            return lambda *a: self.launches.append(name) or 0
        return real(self, name)

    monkeypatch.setattr(type(lib), "__getattr__", entry)
    return g, lib


@pytest.mark.parametrize("M, N, K", [(MORE, 8, 16), (8, MORE, 16), (8, 8, (1 << 32) + 16),
                                     (1 << 31, 8, 16)])
def test_product(all_recorded, M, N, K):
    g, lib = all_recorded
    kb = -(-K // 128)
    with pytest.raises(g.GdrError, match="gdr_product8: .*32 bits"):
        g.gdr_product8(meta(M, K, dtype=E4M3), meta(M, kb, dtype=F32), meta(N, K, dtype=E4M3),
                       meta(-(-N // 128), kb, dtype=F32), meta(M, N))
    assert lib.launches == []


@pytest.mark.parametrize("rows, D, N", [(MORE, 1, 2), (8, MORE, 2), (8, 1, MORE), (1 << 31, 1, 1)])
def test_channels(all_recorded, rows, D, N):
    g, lib = all_recorded
    x, cu, ws = meta(rows, D), meta(N + 1, dtype=torch.int32), meta(1, dtype=torch.uint8)
    with pytest.raises(g.GdrError, match="gdr_channel_prefill: .*32 bits"):
        g.gdr_channel_prefill(x, x, cu, None, None, x, workspace=ws)
    with pytest.raises(g.GdrError, match="gdr_channel_backward: .*32 bits"):
        g.gdr_channel_backward(None, x, x, cu, None, x, None, x, x, workspace=ws)
    if N < 1 << 31 and D * rows < 1 << 62 and max(rows, D) >= 1 << 31:
        with pytest.raises(g.GdrError, match="gdr_channel_decode: .*32 bits"):
            g.gdr_channel_decode(x, x, meta(rows, D, dtype=F32), x)
    assert lib.launches == []


def test_norms(all_recorded):
    g, lib = all_recorded
    D = (1 << 32) + 16
    x = meta(1, D)
    with pytest.raises(g.GdrError, match="gdr_block_norm8: .*32 bits"):
        g.gdr_block_norm8(x, meta(1, D, dtype=E4M3), meta(1, -(-D // 128), dtype=F32))
    with pytest.raises(g.GdrError, match="gdr_block_norm: .*32 bits"):
        g.gdr_block_norm(x, x)
    with pytest.raises(g.GdrError, match="gdr_block_norm_backward: .*32 bits"):
        g.gdr_block_norm_backward(x, x, None, x)
    assert lib.launches == []
