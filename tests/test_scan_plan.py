"""The selective scan's time segments (csrc/scan_plan.h, compiled here as plain C++): for every length that the
calls accept they cover each token once, in order."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rwkv_wkv_recurrence_b200", "csrc")
LONGEST = 2 ** 31 - 1 - 64  # tokens that the calls accept
TILE = 32

SRC = """
#include "scan_plan.h"
using namespace rwkv;
// The tokens that the segments cover from the start without a gap or an overlap; -1 for a plan that has none.
extern "C" int64_t covered(int backward, int64_t tiles, int64_t T, int tile, int algo) {
  const ScanPlan pl = backward ? cut_backward(tiles, T, tile) : cut_forward(tiles, T, tile, algo);
  if (pl.nseg < 1 || pl.seg_len < tile || pl.seg_len % tile != 0) return -1;
  int64_t next = 0;
  for (int s = 0; s < pl.nseg; ++s) {
    if ((int64_t)s * pl.seg_len != next || next >= T) return -1;
    const int end = segment_end((int)T, s * pl.seg_len, pl.seg_len);
    if (end <= next) return next;
    next = end;
  }
  return next;
}
"""


@pytest.fixture(scope="module")
def covered(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    so = str(d / "plan.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", so, str(d / "plan.cpp")])
    f = ctypes.CDLL(so).covered
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int], ctypes.c_int64
    return f


LENGTHS = sorted({t + d for t in (1, 32, 64, 160, 333, 4096, 8192, 1 << 20, 1 << 30, 1 << 31) for d in range(-3, 4)}
                 | {LONGEST - d for d in (0, 1, 31, 32, 100, 1000, 10007, 29630, 29631, 40000, 1000003)})


@pytest.mark.parametrize("tiles", [1, 2, 3, 7, 64, 148, 149, 1000, 5000])
def test_segments_cover_every_token_once(covered, tiles):
    for T in LENGTHS:
        if not 1 <= T <= LONGEST:
            continue
        for backward, algos in ((0, (0, 1, 2)), (1, (0,))):
            for algo in algos:
                assert covered(backward, tiles, T, TILE, algo) == T, (backward, T, algo)
