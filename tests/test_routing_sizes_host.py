"""How the router's kernels share out tokens and slots (csrc/chunks.h), compiled for the
host, up to the largest sizes that the entry points accept."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from swiglu_mlp_gb300 import build as swg_build

MOST = 2 ** 31 - 1024                                    # slots
SOURCE = r"""
#include "chunks.h"
extern "C" void chunk_of(int T, int n, int c, int *out) { swg::chunk_of(T, n, c, out[0], out[1]); }
extern "C" void slots_of_warp(int lo, int hi, int ranking, int warp, int *out)
{
    swg::slots_of_warp(lo, hi, ranking, warp, out[0], out[1]);
}
extern "C" void behind_rows(int rows, int cta, int ctas, int threads, int tid, uint32_t *out)
{
    swg::behind_rows(rows, cta, ctas, threads, tid, out[0], out[1]);
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("chunks")
    src, lib = os.path.join(d, "host.cpp"), os.path.join(d, "host.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-shared", "-fPIC", "-I", swg_build.CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


def two(f, *a, kind=ctypes.c_int):
    out = (kind * 2)()
    f(*a, out)
    return out[0], out[1]


@pytest.mark.parametrize("lo,hi", [(0, 0), (0, 1), (5, 100), (1000, 9193), (7, 5000), (MOST - 1, MOST), (MOST - 8192, MOST),
                                   (MOST - 14128181, MOST), (MOST // 2, MOST), (0, MOST)])
@pytest.mark.parametrize("ranking,warps", [(8, 32), (8, 16), (16, 32), (32, 32), (16, 16)])
def test_warps_share_a_chunk(host, lo, hi, ranking, warps):
    at = lo
    for w in range(warps):
        a, b = two(host.slots_of_warp, lo, hi, ranking, w)
        assert lo <= a <= b <= hi
        assert a == at and (w < ranking or a == b)       # one after the other, nothing left out
        assert b == hi or (b - a) % 32 == 0
        at = b
    assert at == hi


@pytest.mark.parametrize("ctas,threads", [(1, 512), (1, 1024), (152, 1024)])
@pytest.mark.parametrize("slots", [100, 400000, MOST])
def test_places_behind_the_last_row(host, ctas, threads, slots):
    """Each is one thread's, and no thread has any other place."""
    step = ctas * threads
    for rows in {slots, slots - 1, max(slots - step, 0), max(slots - 2 * step - 77, 0)}:
        met = np.zeros(slots - rows, int)
        for cta in range(ctas):
            for tid in range(threads) if ctas == 1 else (0, 1, threads - 1):
                first, by = two(host.behind_rows, rows, cta, ctas, threads, tid, kind=ctypes.c_uint32)
                assert by == step and first == rows + cta * threads + tid
                met[first - rows::by] += 1
        assert (met <= 1).all()
        if ctas == 1:
            assert (met == 1).all()


@pytest.mark.parametrize("T", [0, 1, 7, 8, 9, 63, 64, 65, 5003, 2 ** 30, 1908874354, MOST - 7, MOST])
@pytest.mark.parametrize("per", [8, 64, None])
def test_chunks_share_the_tokens(host, T, per):
    """A CTA for every 8 or 64 tokens, or 152 of a plan."""
    n = 152 if per is None else max(-(-T // per), 1)
    for first, last in ((0, min(n, 300)), (max(n - 300, 0), n)):
        at = min(first * -(-T // n), T)
        for c in range(first, last):
            a, b = two(host.chunk_of, T, n, c)
            assert a == at and a <= b <= T and b - a <= -(-T // n)
            at = b
    assert at == T
