"""The records of the balanced e4m3 decode, on the host: whichever workers give
up, and wherever, every unit that holds tokens has a record written by the
worker whose range it begins in. (The merge behind the decode kernel takes
what it reads and writes from these records, and the workspace that holds
them has no initial value.)  The walk and the cursor are the kernel's own source,
compiled with the host compiler; the loop around them restates the kernel's."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from paged_kv_cache_177_gb300.build import CSRC


def cursor_source():
    """The cursor and its advance, from the kernels' header."""
    with open(os.path.join(CSRC, "pkv_kernels.cuh")) as f:
        text = f.read()
    end = "    c.j += k;\n}\n"
    span = text[text.index("struct Cursor {"):text.index(end) + len(end)]
    return span.replace("__device__ __forceinline__ ", "static ")


SOURCE = r"""
#include "pkv_cursor.cuh"
using namespace pkv;
@CURSOR@
// One worker's range [start, end): its loop up to the block of position start + stop, where it gives up
// (stop = end - start: it does not). written[s * hkv + h] counts the unit's records.
extern "C" void worker(const int *prefix, int S, int hkv, int start, int end, int stop, int *written) {
    const int cnt = end - start;
    if (cnt <= 0) return;
    Cursor c;
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (hkv * prefix[mid] <= start) lo = mid; else hi = mid - 1;
    }
    c.s = lo;
    c.n = prefix[lo + 1] - prefix[lo];
    const int r = start - hkv * prefix[lo];
    c.h = r / c.n;
    c.j = r - c.h * c.n;
    int seg_j0 = c.j, i = 0;
    while (true) {
        if (i == stop) {
            if (seg_j0 == 0) ++written[c.s * hkv + c.h];
            units_begun_later(c, cnt - i, [&](Cursor &at, int k) { cursor_advance(at, k, prefix, hkv); },
                              [&](int s, int h) { ++written[s * hkv + h]; });
            return;
        }
        const bool unit_end = c.j == c.n - 1;
        if (!unit_end && i != cnt - 1) {
            ++c.j, ++i;
            continue;
        }
        if (seg_j0 == 0) ++written[c.s * hkv + c.h];
        if (i == cnt - 1) return;
        ++i;
        cursor_advance(c, 1, prefix, hkv);
        seg_j0 = 0;
    }
}
"""


@pytest.fixture(scope="module")
def worker(tmp_path_factory):
    d = tmp_path_factory.mktemp("cursor")
    src, lib = d / "worker.cpp", d / "worker.so"
    src.write_text(SOURCE.replace("@CURSOR@", cursor_source()))
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)])
    fn = ctypes.CDLL(os.fspath(lib)).worker
    fn.restype = None
    return fn


def ranges(total, workers):
    return [(total * w // workers, total * (w + 1) // workers) for w in range(workers)]


@pytest.mark.parametrize("seed", range(6))
def test_every_unit_is_recorded_wherever_workers_give_up(worker, seed):
    rng = np.random.default_rng(seed)
    hkv = int(rng.choice([1, 3, 8]))
    blocks = rng.integers(0, [2, 4, 9, 30, 3, 60][seed], size=int(rng.integers(1, 12)))
    blocks[rng.integers(len(blocks))] = 40                 # one long unit among the others
    prefix = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32)
    total = hkv * int(prefix[-1])
    held = np.repeat(blocks > 0, hkv)
    p = prefix.ctypes.data_as(ctypes.c_void_p)
    for workers in {1, 2, 3, max(1, total // 4)}:
        whole = np.zeros(len(held), dtype=np.int32)
        for lo, hi in ranges(total, workers):
            ended = np.zeros_like(whole)
            worker(p, len(blocks), hkv, lo, hi, hi - lo, ended.ctypes.data_as(ctypes.c_void_p))
            for stop in range(hi - lo):                    # giving up anywhere records the same units
                got = np.zeros_like(whole)
                worker(p, len(blocks), hkv, lo, hi, stop, got.ctypes.data_as(ctypes.c_void_p))
                assert np.array_equal(got, ended), (workers, lo, hi, stop)
            whole += ended
        assert np.array_equal(whole, held.astype(np.int32))
