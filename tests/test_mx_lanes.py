"""The lanes' reads of the 4-bit few-token product, gone through on the host:
the header the kernel takes its offsets from (csrc/nm_mx_lanes.hpp) compiled
for the CPU."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_structured_sparse_nm_amd", "csrc")

SOURCE = """
#include "nm_mx_lanes.hpp"
extern "C" {
int offset2(int l, int f, int i, int n, int p, int s, int r) { return nm::mx_lane_offset<2>(l, f, i, n, p, s, r); }
int offset4(int l, int f, int i, int n, int p, int s, int r) { return nm::mx_lane_offset<4>(l, f, i, n, p, s, r); }
bool inside2(int l, int i, int s, int r) { return nm::mx_lane_inside<2>(l, i, s, r); }
bool inside4(int l, int i, int s, int r) { return nm::mx_lane_inside<4>(l, i, s, r); }
}
"""


@pytest.fixture(scope="module")
def lanes(tmp_path_factory):
    d = tmp_path_factory.mktemp("lanes")
    (d / "lanes.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "lanes.cpp"), "-o", str(d / "lanes.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "lanes.so"))
    lib.inside2.restype = lib.inside4.restype = ctypes.c_bool
    return lib


@pytest.mark.parametrize("K,eb", [(K, eb) for K in (8, 16, 248, 256, 264, 520, 760) for eb in (2, 4)] + [(12, 4), (516, 4)])
def test_every_lane_reads_inside_its_operand(lanes, K, eb):
    """1 to 16 tokens: no load has a lane outside the rows (a buffer load with
    every lane outside would complete ahead of older ones), and a lane whose
    token and columns exist reads those."""
    offset, inside = (lanes.offset2, lanes.inside2) if eb == 2 else (lanes.offset4, lanes.inside4)
    row = K * eb
    for pitch in (row, row + 48):
        for tokens in range(1, 17):
            for slab in range(0, row, 256 * eb):
                for first in range(0, (tokens + 3) // 4 * 4, 2):
                    for part in range(eb // 2):
                        for lane in range(64):
                            t, col = first + lane // 32, slab + lane % 32 * 8 * eb + 16 * part
                            at = slab + offset(lane, first, part, tokens, pitch, slab, row)
                            assert 0 <= at % pitch and at % pitch + 16 <= row and at // pitch < tokens
                            assert inside(lane, part, slab, row) == (col < row)
                            if t < tokens and col < row:
                                assert at == t * pitch + col
