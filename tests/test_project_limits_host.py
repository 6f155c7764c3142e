"""project= behind a recurrence without a GPU: the product's limits on its rows, and the shapes of
its results (fixtures with recorded launches)."""
import pytest
import torch

from test_norm_after_host import RECURRENCES, host, meta  # noqa: F401
from test_product_host import E4M3, host8, run_after, workspace  # noqa: F401


def norm8(tokens, H, K, F, out=None):
    """Norm in 8 bits of heads of 128 and a product of rows of K values behind it."""
    return dict(h=None, y8=meta(tokens, H, 128, dtype=E4M3),
                y_scale=meta(tokens, H, 1, dtype=torch.float32),
                project=dict(w=meta(F, K, dtype=E4M3),
                             out=meta(*(out or ((tokens, H, F) if K == 128 else (tokens, F)))),
                             w_scale=meta(-(-F // 128), K // 128, dtype=torch.float32)))


# 2^25 rows as long as a head, more than the product takes; 2^24 rows of 4096 results, 2^36 of them;
# 2^23 rows as long as a token of 8192 results, as many
@pytest.mark.parametrize("tokens, H, K, F, rows", [(1 << 20, 32, 128, 64, 1 << 25),
                                                   (1 << 19, 32, 128, 4096, 1 << 24),
                                                   (1 << 23, 4, 512, 8192, 1 << 23)])
@pytest.mark.parametrize("name", RECURRENCES)
def test_rows_that_the_product_refuses_are_refused_before_anything_runs(host8, name, tokens, H, K,  # noqa: F811
                                                                        F, rows):
    g, lib, _ = host8
    with pytest.raises(g.GdrError, match=f"gdr_product8: M={rows}"):
        run_after(g, name, tokens, H, norm8(tokens, H, K, F), **workspace(name))
    assert lib.launches == []


@pytest.mark.parametrize("name", RECURRENCES)
def test_as_many_rows_as_the_product_takes(host8, name):  # noqa: F811
    g, lib, _ = host8
    run_after(g, name, 1 << 19, 32, norm8(1 << 19, 32, 128, 4095), **workspace(name))
    assert [n for n, _, _ in lib.launches] == [name, "gdr_block_norm8", "gdr_product8"]


@pytest.mark.parametrize("decode", [True, False])
def test_the_same_behind_the_recurrence_of_channels(host8, monkeypatch, decode):  # noqa: F811
    g, lib, _ = host8
    real = type(lib).__getattr__

    def entry(self, name):
        if name in ("gdr_channel_decode", "gdr_channel_prefill"):
            return lambda *a: self.launches.append((name, self._current[-1], a[-1])) or 0
        return real(self, name)

    monkeypatch.setattr(type(lib), "__getattr__", entry)

    def step(N, F):
        x, f32 = meta(N, 128), torch.float32
        norm = dict(y8=meta(N, 128, dtype=E4M3), y_scale=meta(N, 1, dtype=f32),
                    project=dict(w=meta(F, 128, dtype=E4M3), out=meta(N, F),
                                 w_scale=meta(-(-F // 128), 1, dtype=f32)))
        if decode:
            g.gdr_channel_decode(x, x, meta(N, 128, dtype=f32), x, norm=norm)
        else:
            g.gdr_channel_prefill(x, x, meta(2, dtype=torch.int32), None, None, x, norm=norm,
                                  workspace=meta(1, dtype=torch.uint8))

    for N, F in ((1 << 25, 64), (1 << 24, 4096)):
        with pytest.raises(g.GdrError, match=f"gdr_product8: M={N}"):
            step(N, F)
        assert lib.launches == []
    step(1 << 20, 64)
    assert [n for n, _, _ in lib.launches] == ["gdr_channel_decode" if decode else "gdr_channel_prefill",
                                               "gdr_block_norm8", "gdr_product8"]


def test_most_rows():
    import gated_delta_rule_100_amd as g
    assert g.gdr_product8_max_rows(1) == g.gdr_product8_max_rows(4095) == 1 << 24
    for N in (4096, 4097, 1 << 20, (1 << 24) - 1, 1 << 24):
        M = g.gdr_product8_max_rows(N)
        assert M * N < 1 << 36 <= (M + 1) * N, N
    assert g.gdr_product8_max_rows(0) == g.gdr_product8_max_rows(-1) == 0
    assert g.gdr_product8_max_rows((1 << 24) + 1) == 0
