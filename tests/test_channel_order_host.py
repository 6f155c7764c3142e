"""Tiles that workgroups of the channel scan take, on the CPU: the header that its kernel takes
them from, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_100_amd", "csrc")
SOURCE = """
#include "channel_order.h"
extern "C" int has(uint32_t ticket, int tiles) { return gdr::has_tile(ticket, tiles); }
extern "C" int tile(uint32_t ticket, int tiles, int back) {
  return gdr::tile_of_ticket(ticket, tiles, back != 0);
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    at = tmp_path_factory.mktemp("order")
    (at / "order.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(at / "order.cpp"), "-o",
                    str(at / "order.so")], check=True)
    lib = ctypes.CDLL(str(at / "order.so"))
    lib.has.argtypes = [ctypes.c_uint32, ctypes.c_int]
    lib.tile.argtypes = [ctypes.c_uint32, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("tiles", [2, 3, 64, 1025])
@pytest.mark.parametrize("back", [0, 1])
def test_tickets_of_one_pass_take_every_tile_once(order, tiles, back):
    assert all(order.has(t, tiles) for t in range(tiles))
    took = [order.tile(t, tiles, back) for t in range(tiles)]
    assert took == (list(range(tiles))[::-1] if back else list(range(tiles)))


@pytest.mark.parametrize("tiles", [1, 2, 1025, 1 << 24])
def test_any_other_ticket_has_no_tile(order, tiles):
    for ticket in (tiles, tiles + 1, 2 * tiles, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) - tiles,
                   (1 << 32) - 1):
        assert not order.has(ticket, tiles), ticket


def test_the_kernel_checks_its_ticket():
    """Before anything is read or written by it."""
    text = open(os.path.join(CSRC, "channel.hip")).read()
    kernel = text[text.index("void channel_scan_kernel"):text.index("void channel_decode_kernel")]
    check = kernel.index("if (!has_tile(ticket, k.tiles)) return;")
    take = kernel.index("tile_of_ticket(order, k.tiles, BACK)")
    assert kernel.index("atomicAdd(k.ticket") < check < take < kernel.index("at_c.load(g[i]")
    assert kernel.count("k.tiles - 1 - ") == 0
