"""The calls with transformed scores refuse bad arguments on the host, before
any launch (no GPU here), and the 64-bit form of their tests is pinned."""
import ctypes

import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_serving_abi import A, ALIGN, ARG, CF, CI, OK, SZ, UNSUPPORTED, VP, WORKSPACE, caller
from paged_kv_cache_177_gb300.build import build_library

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_library())


def test_decode_refusals(lib):
    f = caller(lib, "paged_decode_attention_scored", [
        ("out", VP, A), ("q", VP, A), ("kc", VP, A), ("vc", VP, A), ("bt", VP, A), ("cl", VP, A), ("scale", CF, 0.1),
        ("cap", CF, 30.0), ("win", CI, 7), ("slopes", VP, A), ("hkv", CI, 8), ("S", CI, 4), ("hq", CI, 32), ("d", CI, 128),
        ("maxb", CI, 8), ("nb", CI, 64), ("maxlen", CI, 128), ("dt", CI, 1), ("part", CI, 16), ("ws", VP, None),
        ("wsb", SZ, 0), ("st", VP, None)])
    assert f(cap=-1.0) == ARG and f(cap=NAN) == ARG and f(cap=INF) == ARG and f(win=-1) == ARG
    assert f(cap=1e-44, scale=1e30) == ARG and f(cap=3.3e38) == ARG          # constants past fp32
    assert f(slopes=A + 2) == ALIGN and f(q=A + 8) == ALIGN
    assert f(S=-1) == ARG and f(hkv=0) == ARG and f(hq=33) == ARG and f(maxb=0) == ARG and f(maxlen=-1) == ARG
    assert f(part=-2) == ARG and f(part=17) == ARG and f(scale=NAN) == ARG and f(out=None) == ARG
    assert f(d=96) == UNSUPPORTED and f(hq=8 * 17) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(dt=4) == UNSUPPORTED
    assert f(win=0) == WORKSPACE                                              # 128 tokens in partitions of 16
    assert f(win=100) == WORKSPACE and f(win=100, ws=A, wsb=10240 + 4 * 32 * 8 * 130 * 4 - 1) == WORKSPACE
    assert f(S=0) == OK and f(S=0, slopes=None, cap=0.0, win=0) == OK


def test_prefill_refusals(lib):
    f = caller(lib, "paged_prefill_attention_scored", [
        ("out", VP, A), ("q", VP, A), ("kc", VP, A), ("vc", VP, A), ("bt", VP, A), ("cl", VP, A), ("qs", VP, A),
        ("scale", CF, 0.1), ("cap", CF, 30.0), ("win", CI, 7), ("slopes", VP, A), ("pre", VP, A), ("hkv", CI, 8), ("S", CI, 4),
        ("hq", CI, 32), ("d", CI, 128), ("maxb", CI, 8), ("nb", CI, 64), ("T", CI, 40), ("maxq", CI, 16), ("maxlen", CI, 128),
        ("dt", CI, 1), ("st", VP, None)])
    assert f(cap=-1.0) == ARG and f(cap=NAN) == ARG and f(win=-1) == ARG and f(scale=INF) == ARG
    assert f(S=-1) == ARG and f(hq=33) == ARG and f(T=-1) == ARG and f(maxq=-1) == ARG and f(qs=None) == ARG
    assert f(slopes=A + 2) == ALIGN and f(pre=A + 2) == ALIGN and f(vc=A + 8) == ALIGN
    assert f(dt=0) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(d=80) == UNSUPPORTED and f(hq=8 * 65) == UNSUPPORTED
    assert f(maxq=1 << 30) == UNSUPPORTED and f(nb=1 << 28) == UNSUPPORTED and f(maxb=1 << 28) == UNSUPPORTED
    assert f(S=0) == OK and f(T=0) == OK and f(maxq=0, pre=None, slopes=None) == OK


def test_common_prefix_refusals(lib):
    f = caller(lib, "paged_decode_attention_common_prefix", [
        ("out", VP, A), ("q", VP, A), ("kc", VP, A), ("vc", VP, A), ("bt", VP, A), ("cl", VP, A), ("scale", CF, 0.1),
        ("hkv", CI, 8), ("S", CI, 4), ("hq", CI, 32), ("d", CI, 128), ("maxb", CI, 8), ("nb", CI, 64), ("maxlen", CI, 128),
        ("gs", VP, A), ("sb", VP, A), ("G", CI, 2), ("maxg", CI, 3), ("dt", CI, 1), ("ws", VP, None), ("wsb", SZ, 0),
        ("st", VP, None)])
    assert f(S=-1) == ARG and f(hkv=0) == ARG and f(hq=33) == ARG and f(maxb=0) == ARG and f(maxlen=-1) == ARG
    assert f(G=-1) == ARG and f(maxg=-1) == ARG and f(G=5) == ARG and f(gs=None) == ARG and f(sb=None) == ARG
    assert f(scale=INF) == ARG and f(out=None) == ARG and f(q=A + 8) == ALIGN
    assert f(dt=0) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(d=80) == UNSUPPORTED and f(hq=8 * 17) == UNSUPPORTED
    assert f(S=8193) == UNSUPPORTED and f(nb=1 << 28) == UNSUPPORTED and f(S=4096, maxb=1 << 20, maxlen=1 << 30) == UNSUPPORTED
    assert f() == WORKSPACE and f(ws=A, wsb=1 << 20) == WORKSPACE
    assert f(S=0, G=0) == OK
    g = lib.pkv_common_prefix_workspace_bytes
    g.restype, g.argtypes = SZ, [CI] * 4
    assert g(0, 8, 2, 64) == 0 and g(4, 9, 2, 64) == 0
    assert g(8, 8, 2, 64) - g(4, 8, 2, 64) == 4 * 8 * 66 * 4
    for s in range(1, 70):                     # sums of an odd number of rows are padded to where outputs are aligned
        for hq in (3, 5, 7, 8):
            rest = g(s, hq, 1, 64) - s * hq * 64 * 4
            assert rest % 256 == 0 and rest - (g(1, hq, 1, 64) - hq * 64 * 4) >= s * hq * 8 - 256


def test_the_form_by_hand():
    """Two keys: scores 4 and 0 capped to 2 tanh 2 and 0; a bias of 1 a token; a window that leaves one key."""
    q, k = np.array([[[2.0]]]), np.array([[[2.0]], [[0.0]]])
    v = np.array([[[1.0]], [[0.0]]])
    w = lambda **kw: H.attend(q, k, v, 1.0, [1], **kw)[0][0, 0, 0]
    sig = lambda x: 1 / (1 + np.exp(-x))
    assert np.isclose(w(), sig(4)) and np.isclose(w(cap=2.0), sig(2 * np.tanh(2)))
    assert np.isclose(w(slopes=[1.0]), sig(3)) and w(window=1) == 0.0 and np.isclose(w(window=2), sig(4))
    first = H.attend(np.concatenate([q, q]), k, v, 1.0, [0, 1], prefix=2)[0][0, 0, 0]
    assert np.isclose(first, sig(4)) and H.attend(q, k, v, 1.0, [0])[0][0, 0, 0] == 1.0
    assert H.visible([3], 8, 2, 6).tolist() == [[False, False, True, True, True, False, False, False]]


def test_binding_refuses_bad_tensors():
    B = S.lib()
    q, c = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.paged_decode_attention_scored(q, q, c, c, t, n, 0.1)
