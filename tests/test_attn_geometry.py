"""The attention kernels' integer arithmetic (csrc/qmv_attn_geom.h) built for the host, against
Python's integers: which keys a block of query rows sees, at sizes and windows up to the
largest that the entry accepts."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantized_weight_fly_gb300", "csrc")
INT_MAX = 2 ** 31 - 1

SOURCE = r"""
#include "qmv_attn_geom.h"
using namespace qmv;
extern "C" int first(int pos, int window) { return window_first(pos, window); }
extern "C" void range(int wide, int n, int c, int G, int qb, int causal, int window, int* out) {
  const BlockRange b = wide ? block_range<64, 128>(n, c, G, qb, causal != 0, window)
                            : block_range<128, 256>(n, c, G, qb, causal != 0, window);
  out[0] = b.first_pos; out[1] = b.last_pos; out[2] = b.tile0; out[3] = b.nt; out[4] = b.last;
}
extern "C" int tiles(int tile, int n, int first) { return tile == 32 ? tiles_of<32>(n, first) : tiles_of<16>(n, first); }
extern "C" long long cost(int wide, int n, int c, int G, int lane, int causal, int window, int overhead) {
  const int nqb = (c * G + (wide ? 127 : 255)) / (wide ? 128 : 256);
  return wide ? blocks_cost<64, 128>(n, c, G, nqb, lane, causal != 0, window, overhead)
              : blocks_cost<128, 256>(n, c, G, nqb, lane, causal != 0, window, overhead);
}
"""


def compile_host(tmp, source):
    src, so = os.path.join(tmp, "geom.cpp"), os.path.join(tmp, "geom.so")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.cost.restype = ctypes.c_longlong
    return lib


@pytest.fixture(scope="module")
def geom(tmp_path_factory):
    return compile_host(str(tmp_path_factory.mktemp("geom")), SOURCE)


def block(geom, wide, n, c, G, qb, causal, window):
    out = (ctypes.c_int * 5)()
    geom.range(wide, n, c, G, qb, causal, window, out)
    return list(out)


def first_seen(pos, window):
    return max(0, pos - window + 1) if window else 0


WINDOWS = [0, 1, 2, 63, 64, 65, 128, 1000, 1 << 30, INT_MAX - 1, INT_MAX]


@pytest.mark.parametrize("window", WINDOWS)
def test_first_key_of_a_query(geom, window):
    for pos in (-(1 << 30), -5000, -3, -2, -1, 0, 1, 5, 999, 1000, 1 << 30, INT_MAX - 1):
        assert geom.first(pos, window) == first_seen(pos, window), (pos, window)


@pytest.mark.parametrize("wide,KT,QB", [(0, 128, 256), (1, 64, 128)])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("n,c", [(0, 5), (1, 1), (2, 5), (3, 8), (40, 300), (300, 300), (1000, 77), (5, 1 << 20),
                                 (1 << 20, 900), (INT_MAX - 15, 40)])
def test_keys_of_a_block_of_rows(geom, wide, KT, QB, causal, n, c):
    for window in WINDOWS if causal else [0]:
        for G in (1, 3, 8):
            last_block = (c * G - 1) // QB
            for qb in sorted({0, 1, last_block // 2, last_block}):
                if qb > last_block:
                    continue
                r1 = min((qb + 1) * QB, c * G) - 1
                p0, p1 = n - c + qb * QB // G, n - c + r1 // G
                lo, hi = first_seen(p0, window), p1 if causal else n - 1
                got = block(geom, wide, n, c, G, qb, causal, window)
                assert got[:2] == [p0, p1] and got[4] == hi
                assert got[3] == (0 if hi < lo else hi // KT - lo // KT + 1), (window, G, qb)
                if got[3]:
                    assert got[2] == lo // KT


@pytest.mark.parametrize("wide,KT,QB", [(0, 128, 256), (1, 64, 128)])
@pytest.mark.parametrize("n,c,G,causal,window", [
    (1 << 20, 1 << 20, 16, 0, 0),               # past 2^31 with 64-token tiles: 2^17 blocks of 2^14 + 8
    (3 << 20, 3 << 20, 16, 1, 0),               # a causal triangle past 2^31
    (1 << 20, 1 << 20, 16, 1, 4096),
    (700, 300, 5, 1, 0), (3, 300, 4, 1, 7), (0, 9, 2, 0, 0),
])
def test_cost_of_a_sequence(geom, wide, KT, QB, n, c, G, causal, window):
    over, want = 8, 0
    for qb in range(-(-c * G // QB)):
        r1 = min((qb + 1) * QB, c * G) - 1
        lo, hi = first_seen(n - c + qb * QB // G, window), n - c + r1 // G if causal else n - 1
        want += 0 if hi < lo else hi // KT - lo // KT + 1 + over
    lanes = [geom.cost(wide, n, c, G, lane, causal, window, over) for lane in range(32)]
    assert sum(lanes) == want
    if wide and n >= 1 << 20 and not window:
        assert want > 2 ** 31


@pytest.mark.parametrize("tile", [16, 32])
def test_tiles_of_a_sequence(geom, tile):
    for n in (1, 15, 16, 17, 31, 32, 33, 1000, 2 ** 31 - 48, 2 ** 31 - 17, 2 ** 31 - 16):
        for first in {0, n // 2, n - 1}:
            assert geom.tiles(tile, n, first) == -(-n // tile) - first // tile, (n, first)
