"""The choice of the recurrence's cluster size (csrc/cluster_choice.h), compiled
for the host, with made-up answers of the device."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_sequence_falcon_b200",
                    "csrc")
CODE = """
#include "cluster_choice.h"
using namespace falcon::scan;
static ClustersHeld kept;
extern "C" int choose(long long units, int tiles, const int *held) {
    return choose_cluster(units, tiles, [&](int cs) { return held[cs]; });
}
extern "C" int get(long kernel, int device, int cs, int answer, int *asked) {
    return kept.get(reinterpret_cast<const void *>(kernel), device, cs, [&] { ++*asked; return answer; });
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("cluster")
    (d / "c.cpp").write_text(CODE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I" + CSRC, "c.cpp", "-o", "c.so"], cwd=d, check=True)
    lib = ctypes.CDLL(str(d / "c.so"))
    lib.choose.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    lib.get.argtypes = [ctypes.c_long] + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)]
    return lib


def choose(lib, units, tiles, held):
    return lib.choose(units, tiles, (ctypes.c_int * 17)(0, *[held(cs) for cs in range(1, 17)]))


def fits(cs):  # four blocks on each of 148 SMs
    return 592 // cs


def test_sizes_that_do_not_fit_are_not_taken(lib):
    """One unit takes the largest size there is; never one of which the device
    holds none, or could not say."""
    assert choose(lib, 1, 1000, fits) == 16
    for no in (0, -1):
        assert choose(lib, 1, 1000, lambda cs: no if cs > 8 else fits(cs)) == 8
        assert choose(lib, 1, 1000, lambda cs: no if cs == 16 else fits(cs)) == 15
        assert choose(lib, 1, 1000, lambda cs: no if cs > 1 else fits(cs)) == 1
        assert choose(lib, 300, 40, lambda cs: no) == 1


def test_no_more_blocks_than_tiles(lib):
    assert [choose(lib, 1, tiles, fits) for tiles in (0, 1, 2, 3, 16, 10 ** 6)] == [1, 1, 2, 3, 16, 16]
    assert choose(lib, 10 ** 9, 1, fits) == 1


def test_answers_are_kept_and_failures_are_not(lib):
    asked = ctypes.c_int(0)
    get = lambda kernel, dev, cs, answer: lib.get(kernel, dev, cs, answer, ctypes.byref(asked))  # noqa: E731
    assert get(1, 0, 4, -1) == -1 and get(1, 0, 4, -1) == -1 and asked.value == 2   # could not be asked: asked again
    assert get(1, 0, 4, 7) == 7 and get(1, 0, 4, 9) == 7 and asked.value == 3
    assert get(1, 0, 16, 0) == 0 and get(1, 0, 16, 5) == 0 and asked.value == 4     # none fits: known
    assert get(1, 1, 4, 8) == 8 and get(2, 0, 4, 6) == 6 and get(1, 0, 5, 3) == 3 and asked.value == 7
    assert get(1, 99, 4, 2) == 2 and get(1, 99, 4, 3) == 3 and get(1, -1, 4, 1) == 1  # devices beyond the table
    for kernel in range(100, 200):                                                     # and kernels
        assert get(kernel, 0, 1, 11) == 11
    assert get(1, 0, 4, 1) == 7
