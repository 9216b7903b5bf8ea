"""The launches that rows in 8 bits are divided into, by the library's own rule compiled for the host: they cover every
row once, stay below HIP's 2^32 threads, and find each block's row by their product and shift."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bounded_expert_amd", "csrc")


class Launch(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64)] + [(n, ctypes.c_uint32) for n in ("units", "groups", "magic", "shift")]


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches(N, blocks) -> the launches of N rows."""
    d = tmp_path_factory.mktemp("q8")
    src, lib = str(d / "s.cpp"), str(d / "s.so")
    open(src, "w").write('#include "q8_shapes.hpp"\nextern "C" {\n'
                         "moe::Q8Launch next(int64_t left, int blocks) { return moe::q8_launch(left, blocks); }\n"
                         "int threads() { return moe::kQ8GroupThreads; }\nint per_group() { return moe::kQ8GroupBlocks; }\n}\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", src, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.next.argtypes, L.next.restype = [ctypes.c_int64, ctypes.c_int], Launch
    assert L.threads() == 8 * L.per_group()

    def of(N, blocks):
        out, left = [], N
        while left > 0:
            out.append(L.next(left, blocks))
            assert out[-1].rows > 0
            left -= out[-1].rows
        assert left == 0
        return out, L.threads(), L.per_group()

    return of


EDGE = (1 << 29) - 32  # the most blocks of a launch


@pytest.mark.parametrize("N", [1, 31, 33, EDGE // 512, EDGE // 512 + 1, EDGE - 1, EDGE, EDGE + 1, 540_000_000, 600_000_000, (1 << 31) - 1])
@pytest.mark.parametrize("blocks", [1, 2, 3, 7, 12, 16, 100, 511, 512])
def test_launches_are_ones_that_hip_takes(launches, N, blocks):
    every, threads, per_group = launches(N, blocks)
    assert sum(l.rows for l in every) == N
    for l in every:
        assert l.units == l.rows * blocks <= l.groups * per_group < l.units + per_group
        assert l.groups * threads < 1 << 32
        for row in (0, 1, l.rows // 3, l.rows - 2, l.rows - 1):
            for u in (row * blocks, row * blocks + blocks - 1):
                if 0 <= u < l.units:
                    assert u * l.magic < 1 << 64 and u * l.magic >> l.shift == u // blocks
    assert len(every) == 1 or all(l.groups * threads > (1 << 32) - 2 * 512 * 256 for l in every[:-1])


def test_rows_past_a_launch_are_another(launches):
    assert len(launches(EDGE, 1)[0]) == 1 and [l.rows for l in launches(EDGE + 1, 1)[0]] == [EDGE, 1]
