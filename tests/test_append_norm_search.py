"""The search for a row's sequence in the normalising writer (extend.cuh lane_find_sequence), compiled from the product header
for the host with loads that check their place: right for every ascending array, inside the array for any."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(HERE, "..", "mixed_precision_paged_gb300", "csrc", "extend.cuh")

HARNESS = """
#include <algorithm>
#include <cstdint>
using std::max;
using std::min;
#define __device__
#define __forceinline__ inline
static const int32_t* array;
static int count, outside;
static int __ldg(const int32_t* p) {
  const long long at = ((intptr_t)p - (intptr_t)array) / 4;
  if (at < 0 || at >= count) return ++outside, 0;
  return array[at];
}
%s
extern "C" int find(const int32_t* cu, int batch, int i, int first, int last, int* b) {
  array = cu, count = batch + 1, outside = 0;
  *b = lane_find_sequence(cu, batch, i, first, last);
  return outside;
}
"""


@pytest.fixture(scope="module")
def find(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    text = open(HEADER).read()
    at = text.index("__device__ __forceinline__ int lane_find_sequence")
    tmp = tmp_path_factory.mktemp("search")
    src, lib = str(tmp / "search.cpp"), str(tmp / "search.so")
    with open(src, "w") as f:
        f.write(HARNESS % text[at:text.index("\n}\n", at) + 3])
    subprocess.run([cxx, "-O1", "-fwrapv", "-std=c++17", "-shared", "-fPIC", src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).find

    def call(cu, i, last):
        """(sequence, reads outside cu) of row i, the rows running from cu[0] to `last`, as the writer asks."""
        b = ctypes.c_int(-1)
        out = fn(cu.ctypes.data_as(ctypes.c_void_p), len(cu) - 1, i, int(cu[0]), last, ctypes.byref(b))
        return b.value, out
    return call


def test_ascending_arrays(find):
    rng = np.random.default_rng(400)
    for batch in (1, 2, 3, 8, 9, 33, 300):
        for top in (1, 2, 40):
            new = rng.integers(0, top + 1, batch) * (rng.random(batch) < rng.choice([0.1, 0.9]))
            new[rng.integers(batch)] = 7 * top
            cu = (np.cumsum([0] + list(new)) + rng.choice([0, 5])).astype(np.int32)
            want = np.searchsorted(cu[1:], np.arange(cu[0], cu[-1]), side="right")
            got = [find(cu, i, int(cu[-1])) for i in range(cu[0], cu[-1])]
            assert got == [(int(b), 0) for b in want]


@pytest.mark.parametrize("low", [-1, -5, -2 ** 30, -2 ** 31 + 4, -2 ** 31 + 100, -2 ** 31])
def test_a_first_row_below_zero(find, low):
    """Row 0 and those behind it belong to the sequence that begins there, which fails its checks; the others to theirs."""
    for batch in (1, 4, 40):
        cu = np.arange(0, 3 * batch + 1, 3, dtype=np.int32)
        cu[0] = low
        for i in range(3 * batch):
            assert find(cu, i, 3 * batch) == (i // 3, 0)


def test_any_array_is_read_inside(find):
    """Arrays of anything: no read outside, and a sequence that ends behind the row or begins behind it (and fails)."""
    rng = np.random.default_rng(401)
    ends = np.array([-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 9, -9, -1, 0, 1, 9, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1])
    for _ in range(3000):
        batch = int(rng.integers(1, 30))
        kind = rng.integers(3)
        cu = (rng.choice(ends, batch + 1) if kind == 0 else rng.integers(-2 ** 31, 2 ** 31, batch + 1) if kind == 1
              else rng.integers(-5, 30, batch + 1)).astype(np.int32)
        last = min(int(rng.choice([20, 2 ** 31 - 1])), int(cu[-1]))
        for i in {0, 1, 5, last // 2, last - 1}:
            if not max(0, int(cu[0])) <= i < last:         # (the writer asks for such rows alone)
                continue
            b, out = find(cu, i, last)
            assert out == 0 and 0 <= b < batch and (i < cu[b] or i < cu[b + 1]), (cu.tolist(), i, last)
