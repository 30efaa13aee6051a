"""Caps far above what a model's scores reach, with scores that reach them all
the same: equal scores weigh the same wherever they lie, but for the errors of
the two forms of the cap."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_gpu_scored_prefill import i32, make

pytestmark = pytest.mark.gpu
bf16 = lambda x: float(torch.tensor(x, dtype=torch.bfloat16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [50.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("part", [0.74, 0.3, 0.1, 0.04, 1e-6])
def test_equal_scores_in_two_places(part, cap, d):
    """Row 0 scores two tokens, of two chunks, at this part of the cap, and the others next to nothing; row 1 one beside
    the second at 0.95 of it."""
    B = S.lib()
    q, k, v, tables, kr, vr, start = make(17, [700], [2], 1, 1, d)
    tb = tables.cpu().numpy()
    at, scale = bf16(cap ** 0.5), 0.0884
    k *= 0.01
    kr[0][:] = S.f64(k)[tb[0, np.arange(700) // 16], :, np.arange(700) % 16]
    q[:2] = 0.0
    for t, e in ((5, 0), (300, 0), (310, 1)):
        k[tb[0, t // 16], 0, t % 16] = 0.0
        k[tb[0, t // 16], 0, t % 16, e] = at
        kr[0][t] = 0.0
        kr[0][t, 0, e] = at
    q[0, 0, 0], q[1, 0, 1] = part * cap / (at * scale), 0.95 * cap / (at * scale)
    out = torch.empty_like(q)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32([700]), i32(start), scale, softcap=cap)
    # The bound: the roundings of the output and of the weights, and the scores' errors. A score below three quarters of the
    # cap may be taken by a polynomial, 5.7e-7 of it off and a few fp32 roundings, or as those above it, 2^-20 of it
    # off; which, is decided 64 columns at a time. So two tokens of one score are weighed up to d = 2^-19 of it
    # apart, and every weight and the sum change by e^d at most. (From caps of 10^6 on that leaves the values' range only.)
    qf = S.f64(q[:2])
    got = S.f64(out[:2])
    for row in range(2):
        want, _ = H.attend(qf[row:row + 1], kr[0], vr[0], scale, [698 + row], cap)
        raw = kr[0][:699 + row, 0] @ qf[row, 0] * scale
        x = cap * np.tanh(raw / cap)
        p = np.exp(x - x.max())
        p /= p.sum()
        v = np.abs(vr[0][:699 + row, 0])
        d = np.expm1(min(2 * np.abs(x).max() * 2.0 ** -19, 50.0)) if row == 0 else 0.0     # (row 1: one token)
        spread = p @ v
        bound = np.minimum(2.0 ** -8 * np.abs(want[0, 0]) + (2 * 2.0 ** -8 + d) * spread, 2.02 * v.max(0)) + 1e-6
        assert np.all(np.abs(got[row, 0] - want[0, 0]) <= bound), (row, np.abs(got[row, 0] - want[0, 0]).max())
