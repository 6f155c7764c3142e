"""project= behind a recurrence of one head without a GPU: rows of w are then as long as the head
and as all heads of a token, and out may have either shape."""
import pytest

from test_norm_after_host import RECURRENCES, host, meta  # noqa: F401
from test_product_host import host8, run_after, workspace  # noqa: F401
from test_project_limits_host import norm8


@pytest.mark.parametrize("out", [(128, 96), (128, 1, 96)])
@pytest.mark.parametrize("name", RECURRENCES)
def test_both_shapes_of_one_head(host8, name, out):  # noqa: F811
    g, lib, _ = host8
    run_after(g, name, 128, 1, norm8(128, 1, 128, 96, out), **workspace(name))
    assert [n for n, _, _ in lib.launches] == [name, "gdr_block_norm8", "gdr_product8"]


@pytest.mark.parametrize("H, K, out", [(1, 128, (128, 95)), (1, 128, (96,)), (1, 128, (1, 128, 96)),
                                       (4, 128, (128, 96)), (4, 512, (128, 4, 96))])
@pytest.mark.parametrize("name", RECURRENCES)
def test_other_shapes(host8, name, H, K, out):  # noqa: F811
    g, lib, _ = host8
    with pytest.raises(g.GdrError, match="out must have shape"):
        run_after(g, name, 128, H, norm8(128, H, K, 96, out), **workspace(name))
    assert lib.launches == []
