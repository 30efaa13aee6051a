"""Slopes so steep that a bias passes fp32: all of a row's weight is at its own
position, or for a negative slope at the farthest that it sees."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_gpu_scored_prefill import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()
STEEP = np.array([3.4e38, 1e36, -3.4e38, 1e30, -1e36, 2e34, 1e25, -1e25], dtype=np.float32)


def check(got, v, rows, slopes, step=0.0):
    """Row i of got [n, Hq, D] against the value at rows[i] = (nearest, farthest), whose weight is 1: every other token
    lies 10^25 below in the exponent, 10^25 past any score here.  step: of the two tf32 parts (11 bits each, so up to
    2^-21 of it left out) that the fp32 form's tensor cores take of a value; else the value comes out as it is."""
    g = len(slopes) // v.shape[1]
    for i, (near, far) in enumerate(rows):
        for h, x in enumerate(slopes):
            want = v[near if x > 0 else far, h // g]
            assert np.all(np.abs(got[i, h] - want) <= step * np.abs(want)), (i, h, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hkv", [8, 4, 1])
@pytest.mark.parametrize("parts", [0, 64, -1])
@pytest.mark.parametrize("cap,window", [(0.0, 0), (30.0, 0), (0.0, 100)])
def test_decode(cap, window, parts, hkv, dtype):
    if dtype == F32 and parts < 0:
        parts = 512
    B = S.lib()
    B.device_error()
    lens = [1, 2, 17, 64, 65, 300, 2000, 700]
    k, v, tables, _, vr = H.paged(3, lens, hkv, 64, dtype, window)
    q = torch.randn(len(lens), 8, 64, device="cuda").to(dtype)
    out = torch.full_like(q, 55.0)
    B.paged_decode_attention_scored(out, q, k, v, tables, i32(lens), 0.125, softcap=cap, window=window,
                                    slopes=torch.from_numpy(STEEP).cuda(), partition_tokens=parts)
    for s, n in enumerate(lens):
        check(S.f64(out[s:s + 1]), vr[s], [(n - 1, max(0, n - window) if window else 0)], STEEP,
              2.0 ** -20 if dtype == F32 and hkv == 1 else 0.0)
    assert B.device_error() == 0


@pytest.mark.parametrize("hkv", [8, 2])
@pytest.mark.parametrize("cap,window,prefix", [(0.0, 0, False), (30.0, 0, False), (0.0, 100, False), (9.0, 0, True), (0.0, 70, True)])
@pytest.mark.parametrize("lens,ns", [([3000], [5]), ([300, 129, 17, 1], [300, 60, 17, 1])])
def test_prefill(lens, ns, cap, window, prefix, hkv):
    B = S.lib()
    B.device_error()
    q, k, v, tables, _, vr, start = make(5, lens, ns, 8, hkv, 64, window)
    out = torch.full_like(q, 55.0)
    pre = [n * 2 // 3 for n in lens] if prefix else [0] * len(lens)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32(start), 0.125, softcap=cap, window=window,
                                     slopes=torch.from_numpy(STEEP).cuda(), prefix_lens=i32(pre) if prefix else None)
    for s, n in enumerate(lens):
        rows = []
        for pos in range(n - ns[s], n):
            see = np.flatnonzero(H.visible([pos], n, window, pre[s])[0])
            first, last = see[0], see[-1]
            rows.append((pos, first if pos - first >= last - pos else last))
            if pos - first == last - pos and first != last:
                rows[-1] = None                           # (two farthest)
        got = S.f64(out[start[s]:start[s + 1]])
        keep = [i for i, r in enumerate(rows) if r is not None]
        check(got[keep], vr[s], [rows[i] for i in keep], STEEP)
    assert B.device_error() == 0
