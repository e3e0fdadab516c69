"""Which tiles the e4m3 product takes, from its sizes: the rule alone, compiled for the host."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_moe_router_gb300", "csrc")
SHIM = """
#include "qs_fp8tiles.h"
extern "C" void pick(int rows, int cols, int experts, int grouped, int n_sm, int wide, long long *out) {
    const qs::MmTiles t = qs::pick_tiles(rows, cols, experts, grouped != 0, n_sm, wide != 0);
    out[0] = t.cols, out[1] = t.pair, out[2] = t.few, out[3] = t.count;
}
"""


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, "-o", str(d / "shim.so"), str(d / "shim.cpp")], check=True)
    fn = ctypes.CDLL(str(d / "shim.so")).pick

    def call(rows, cols, experts=0, n_sm=152, wide=True):
        out = (ctypes.c_longlong * 4)()
        fn(rows, cols, max(experts, 1), experts > 0, n_sm, wide, out)
        return tuple(out)

    return call


def sizes():
    r = random.Random(1)
    log = lambda lo, hi: int(2 ** r.uniform(lo, hi))  # noqa: E731
    return [(log(0, 18), log(0, 16), r.choice([0, 0, log(0, 10)])) for _ in range(3000)] + [(1 << 30, 1 << 30, e) for e in (0, 1, 1024)]


def test_every_size_has_tiles_that_cover_it(pick):
    for rows, cols, experts in sizes():
        for wide in (True, False):
            width, pair, few, count = pick(rows, cols, experts, wide=wide)
            assert (width, few) in {(16, 0), (32, 0), (64, 0), (128, 0), (256, 0), (64, 16), (128, 16), (64, 32)} and (not pair or width == 256)
            high = 256 if pair else few or 128
            assert count >= -(-cols // width) * (-(-rows // high) if not experts else min(rows, experts))


def test_without_the_widest_tiles_the_others_take_every_size(pick):
    """Tiles of 256 weight rows need a launch with a certain number of registers; a build without it still multiplies."""
    seen = set()
    for rows, cols, experts in sizes():
        width, pair, few, _ = pick(rows, cols, experts, wide=False)
        assert width <= 128 and not pair
        if pick(rows, cols, experts)[0] < 256:
            assert pick(rows, cols, experts, wide=False) == pick(rows, cols, experts)
        seen.add((width, few))
    assert len(seen) == 7
    assert pick(8192, 8192, wide=False) == (128, 0, 0, 64 * 64)


def test_tiles_of_ordinary_sizes(pick):
    assert pick(8192, 8192)[:3] == (256, True, 0)
    assert pick(1, 4096) == (64, False, 16, 64)
    assert pick(200, 1024)[:3] == (64, False, 32)
    assert pick(1, 20000)[:3] == (128, False, 16)
    assert pick(64, 1024, 256)[:3] == (128, False, 16)
    assert pick(8, 512, 256)[:3] == (64, False, 16)
    assert pick(16384, 1024, 256)[:3] == (256, False, 0)
