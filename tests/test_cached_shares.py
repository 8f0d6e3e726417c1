"""How the attention over a paged cache is divided among the CTAs (csrc/shares.cuh), checked on the host: every key
tile of every unit is in one part, every part that a join counts is written in the same call and every part that is
written is joined, whatever the lengths and however coarsely the costs are counted."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "feed_forward_view_vggt_b200", "csrc")
SINGLE, PAIR, FEW = 0, 1, 2


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("shares") / "shares.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    CSRC, "-o", lib, os.path.join(HERE, "shares_host.cpp")], check=True)
    fn = ctypes.CDLL(lib).walk
    i32 = np.ctypeslib.ndpointer(np.int32, flags="C")
    fn.argtypes, fn.restype = [ctypes.c_int, i32, i32, ctypes.c_int, ctypes.c_int], ctypes.c_int
    return lambda kinds, tiles, shift, grid=148: fn(len(kinds), np.array(kinds, np.int32), np.array(tiles, np.int32),
                                                    shift, grid)


@pytest.mark.parametrize("shift", range(13))
def test_random_batches(walk, shift):
    rng = np.random.default_rng(shift)
    for _ in range(2000):
        heads = int(rng.choice([1, 2, 3, 8, 16, 64]))
        units, tiles = [], []
        for _ in range(int(rng.integers(1, 12))):  # sequences: pairs of like or rising length, then a last unit
            most = int(np.exp(rng.uniform(0, np.log(4000)))) if rng.random() < 0.8 else 0
            pairs = int(rng.choice([0, 0, 1, 3, 9]))
            own = [PAIR] * pairs + [int(rng.choice([SINGLE, FEW, PAIR]))]
            of = sorted(int(x) for x in rng.integers(0, most + 1, len(own))) if rng.random() < 0.5 else [most] * len(own)
            units += own * heads
            tiles += of * heads
        grid = int(rng.choice([148, 148, 132, 20, 1]))
        assert walk(units, tiles, shift, grid) == 0, (units, tiles, grid)


@pytest.mark.parametrize("heads,tiles,kind,shift", [(64, 3, FEW, 2), (64, 5, FEW, 2), (16, 20, PAIR, 3), (16, 5, FEW, 4),
                                                    (16, 16, FEW, 4), (32, 16, FEW, 4), (1, 2000, PAIR, 10),
                                                    (64, 16, SINGLE, 2)])
def test_little_work_in_buffers_of_full_size(walk, heads, tiles, kind, shift):
    # fewer points than CTAs: no share between two parts of a unit may be empty
    assert walk([kind] * heads, [tiles] * heads, shift) == 0


def test_the_line_of_a_large_batch(walk):
    rng = np.random.default_rng(1)
    tiles = rng.integers(0, 3, 4096 * 16)
    assert walk(rng.choice([SINGLE, PAIR, FEW], 4096 * 16), tiles, 0) == 0
    assert walk([PAIR] * 96, [1085] * 96, 0) == 0
