"""Sizes that the launches of linear attention cannot hold are refused before a device is touched."""
from test_linear_host import FAKE, _call, lib  # noqa: F401


def test_shared_heads_that_one_launch_cannot_sum_are_refused(lib):  # noqa: F811
    at = dict(N=1, T=1 << 21, H=128, Hk=64, dk=128, ws=FAKE, wsb=1 << 62)
    assert _call(lib, "backward", at) == 1
    assert "shared heads" in lib.gdr_last_error().decode()
    # heads of their own, and just within the limit: refused for the workspace alone
    for over in (dict(Hk=128), dict(T=(1 << 21) - 1)):
        assert _call(lib, "backward", dict(at, wsb=64, **over)) == 1
        assert "workspace" in lib.gdr_last_error().decode()
