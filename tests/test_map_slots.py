"""Where the encoded tensor maps of an array are kept: those that one call takes, and those of both
kernels that take turns on a matrix, do not put one another out."""
import ctypes
import os
import random
import subprocess

import pytest

SOURCE = """
#include "q4k_maps.h"
extern "C" unsigned slot(unsigned long long ptr, long long a, long long b, int box, int kind) {
    return q4k::map_slot_index(q4k::MapKey{static_cast<uintptr_t>(ptr), a, b, box, kind});
}
extern "C" int slots() { return q4k::kMapCacheSize; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from gguf_q4_dequant_gb300 import build
    d = tmp_path_factory.mktemp("maps")
    src, out = str(d / "slots.cpp"), str(d / "slots.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{build.CSRC}", src, "-o", out], check=True)
    assert os.path.exists(out)
    L = ctypes.CDLL(out)
    L.slot.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    L.slot.restype = ctypes.c_uint
    return L


def arrays(n):
    rng = random.Random(5)
    for _ in range(n):
        yield 0x7F0000000000 + 512 * rng.randrange(1 << 30), rng.choice([1, 48, 512, 16384, 32768, 98304]), 256 * rng.randrange(1, 64)


def test_boxes_of_an_array(lib):
    for ptr, rows, K in arrays(500):
        assert len({lib.slot(ptr, rows, K, 32 * i, 2) for i in range(1, 7)}) == 6             # rows of x, many an expert
        assert len({lib.slot(ptr, rows, K, box, 0) for box in (32, 128)}) == 2                # weights, few and many
        assert len({lib.slot(ptr, rows, K, 32 << i, kind) for i in range(4) for kind in (1, 2)}) == 8


def test_arrays_are_spread(lib):
    """As many arrays as a model has matrices: a slot holds few of them."""
    n = lib.slots()
    count = [0] * n
    for ptr, rows, K in arrays(n):
        s = lib.slot(ptr, rows, K, 128, 0)
        assert 0 <= s < n
        count[s] += 1
    # n balls in n slots: 1/e of them empty, the fullest with some ln n / ln ln n
    assert sum(c > 0 for c in count) > 0.55 * n and max(count) <= 10
