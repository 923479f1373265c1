"""The offset checks that the kernels make before they use an expert's rows (csrc/expert_rows.h), on the CPU."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from moe_prefill_nvfp4_gb300 import build

TOP, LOW = 2 ** 31 - 1, -(2 ** 31)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    d = tmp_path_factory.mktemp("expert_rows")
    src, so = d / "t.cpp", d / "t.so"
    src.write_text('#include "expert_rows.h"\n'
                   'extern "C" int rows_ok(int lo, int hi, int R) { return moe::expert_rows_ok(lo, hi, R); }\n'
                   'extern "C" int tiles(int rows, int per) { return moe::tiles_of_rows(rows, per); }\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-shared", "-Wall", "-Werror", "-I", build.CSRC, str(src),
                    "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def wraps(offsets):
    """Whether the steps' 32-bit differences are all at least 0 although the sequence is not what it should be."""
    with np.errstate(over="ignore"):
        return bool((np.diff(np.array(offsets, np.int32)) >= 0).all())


@pytest.mark.parametrize("offsets", [
    [0, 2 ** 30, LOW + 5, -1000, 100],  # 2^30 down to -2^31 + 5 is a step of 2^30 + 5 in 32 bits
    [0, TOP, LOW, -1, 8],
    [0, 2 ** 30, LOW, LOW + 2 ** 30, 0],
    [0, 2 * 10 ** 9, -2 * 10 ** 9, 100],
])
def test_sequences_that_wrap_are_refused(L, offsets):
    assert wraps(offsets)  # a check of the differences' sign, of the first and of the last offset would pass
    assert 0 <= offsets[-1] <= 100
    assert not all(L.rows_ok(a, b, 100) for a, b in zip(offsets, offsets[1:]))


def test_steps(L):
    edge = [LOW, LOW + 1, -2, -1, 0, 1, 2, 99, 100, 101, 2 ** 30, TOP - 1, TOP]
    for R in (0, 1, 100, TOP):
        for lo in edge:
            for hi in edge:
                assert bool(L.rows_ok(lo, hi, R)) == (0 <= lo <= hi <= R), (lo, hi, R)


def test_tiles(L):
    for per in (16, 32, 128):
        for rows in (0, 1, per - 1, per, per + 1, 10 * per + 3, TOP - 1, TOP):
            assert L.tiles(rows, per) == -(-rows // per), (rows, per)
