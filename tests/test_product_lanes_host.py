"""Which bytes the product of few rows loads, on the CPU: the header that its kernel takes the
offsets from, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_100_amd", "csrc")
SOURCE = """
#include "product_lanes.h"
extern "C" int offset(int K, int b, int q, int half) { return gdr::lane_offset(K, b, q, half); }
extern "C" int has(int K, int b, int q, int half) { return gdr::lane_has(K, b, q, half); }
"""


@pytest.fixture(scope="module")
def lanes(tmp_path_factory):
    at = tmp_path_factory.mktemp("lanes")
    (at / "lanes.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(at / "lanes.cpp"), "-o",
                    str(at / "lanes.so")], check=True)
    return ctypes.CDLL(str(at / "lanes.so"))


@pytest.mark.parametrize("K", range(16, 528, 16))
def test_every_load_is_inside_its_row_and_every_value_is_loaded_once(lanes, K):
    taken = []
    for b in range(-(-K // 128)):
        for q in range(4):
            for half in range(2):
                at = lanes.offset(K, b, q, half)
                assert 0 <= at and at + 16 <= K and at % 16 == 0, (b, q, half, at)
                if lanes.has(K, b, q, half):
                    taken.append(at)
    assert sorted(taken) == list(range(0, K, 16))


def test_the_kernel_takes_its_offsets_from_the_header():
    """Rows' pointers hold nothing of a lane's own, and what is loaded is a row's pointer and an
    offset of lane_offset."""
    text = open(os.path.join(CSRC, "product.hip")).read()
    kernel = text[text.index("void product8_rows_kernel"):text.index("hipError_t launch_tiles")]
    assert "q * 16" not in kernel
    assert kernel.count("lane_offset(p.K, b, q,") == 2
