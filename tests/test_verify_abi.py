"""verify_drafts refuses bad arguments on the host, before any launch (no GPU
here), and the binding refuses bad tensors; the walk its GPU tests use is
pinned."""
import ctypes

import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests import verify_helpers as V
from tests.test_serving_abi import ALIGN, ARG, CI, I64, OK, OVERLAP, UNSUPPORTED, VP, caller
from paged_kv_cache_177_gb300.build import build_library

A = 1 << 20                                   # aligned addresses that nothing reads, far apart


@pytest.fixture(scope="module")
def f():
    return caller(ctypes.CDLL(build_library()), "verify_drafts", [
        ("acc", VP, A), ("most", CI, 4), ("num", VP, 2 * A), ("next", VP, 3 * A), ("tok", VP, 4 * A), ("par", VP, 5 * A),
        ("qs", VP, 6 * A), ("p", VP, 7 * A), ("ps", I64, 100), ("q", VP, 8 * A), ("ds", I64, 100), ("u", VP, 9 * A),
        ("fu", VP, 10 * A), ("S", CI, 2), ("T", CI, 8), ("maxq", CI, 5), ("v", CI, 100), ("dt", CI, 0), ("st", VP, None)])


def test_bad_sizes_and_pointers(f):
    assert f(S=-1) == ARG and f(T=-1) == ARG and f(maxq=-1) == ARG and f(most=0) == ARG and f(v=0) == ARG
    assert f(ps=99) == ARG and f(ds=99) == ARG
    for name in ("acc", "num", "next", "tok", "par", "qs", "p", "u", "fu"):
        assert f(**{name: None}) == ARG
    assert f(dt=2) == UNSUPPORTED and f(dt=4) == UNSUPPORTED and f(maxq=1025) == UNSUPPORTED
    assert f(v=(1 << 30) + 1, ps=1 << 31, ds=1 << 31) == UNSUPPORTED and f(ps=1 << 62) == UNSUPPORTED
    assert f(S=(1 << 24) + 1) == UNSUPPORTED
    assert f(S=0) == OK and f(S=0, acc=None) == OK


def test_alignment_is_that_of_the_elements(f):
    for name, off in (("acc", 2), ("num", 2), ("next", 4), ("tok", 4), ("par", 2), ("qs", 2), ("p", 2), ("q", 2), ("u", 2),
                      ("fu", 2)):
        base = {"acc": 1, "num": 2, "next": 3, "tok": 4, "par": 5, "qs": 6, "p": 7, "q": 8, "u": 9, "fu": 10}[name] * A
        assert f(**{name: base + off}) == ALIGN


def test_outputs_over_inputs_and_each_other(f):
    assert f(acc=2 * A - 4) == OVERLAP and f(acc=3 * A - 28) == OVERLAP and f(num=3 * A + 8) == OVERLAP
    for name, at in (("tok", 4), ("par", 5), ("qs", 6), ("p", 7), ("q", 8), ("u", 9), ("fu", 10)):
        assert f(acc=at * A) == OVERLAP and f(num=at * A + 4) == OVERLAP and f(next=at * A - 8) == OVERLAP
    assert f(num=7 * A + (7 * 100 + 99) * 4) == OVERLAP          # the last probability
    assert f(num=8 * A + (7 * 100 + 99) * 4) == OVERLAP


def test_the_walk_by_hand():
    """p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4): the draft 1 stands below u = 1/2, and refused leaves (1, 0, 0)."""
    p, q = np.array([[0.5, 0.25, 0.25]] * 2), np.array([[0.25, 0.5, 0.25]] * 2)
    go = lambda u, final, draft=q: V.walk(2, [-1, 0], [0, 1], p, draft, [0, u], final, 4)
    assert go(0.49, 0.6) == ([0, 1], 1) and go(0.5, 0.6) == ([0], 0) and go(0.5, 0.99) == ([0], 0)
    assert go(0.24, 0.0, None) == ([0, 1], 0) and go(0.25, 0.7, None) == ([0], 2) and go(0.25, 0.66, None) == ([0], 0)


def test_binding_refuses_bad_tensors():
    B = S.lib()
    cpu = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.verify_drafts(cpu, cpu[0], cpu[0].long(), cpu[0].long(), cpu[0], cpu[0], torch.zeros(4, 8), torch.zeros(4),
                        torch.zeros(2))
