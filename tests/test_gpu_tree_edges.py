"""Tree attention where a row's few keys or a draft's non-finite values decide
the answer: weights of rows that see few keys keep their remainders wherever
the keys lie, and an infinity or NaN in a draft's value shows in that element
of the rows that see it, and nowhere else."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests.test_gpu_tree import Case, attend

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -8                                # the output's, to bf16


@pytest.mark.parametrize("ctx,n", [(0, 100), (1, 300), (3, 520), (2, 1000), (60, 400)])
@pytest.mark.parametrize("hkv,g,d", [(2, 1, 128), (1, 4, 64), (1, 8, 128)])
@pytest.mark.parametrize("most_ctx", [None, 4096])
def test_rows_of_few_keys_keep_sixteen_bits_of_their_weights(ctx, n, hkv, g, d, most_ctx):
    """A flat tree: each draft sees the context, itself and at most two earlier drafts. Beside the output's rounding
    a row may be off by sum p |v| times 2^-16 for the weights and 2^-13 for the scores: 128 terms in fp32 with
    sum |q k| scale below 16, and 2^x within 2^-22. (Weights of one bf16 each are off by up to 2^-9 of it.)"""
    b = S.lib()
    rng = np.random.default_rng(n + d)
    see = np.eye(n, dtype=bool)
    for i in range(1, n):
        see[i, rng.integers(0, i, size=2 if ctx < 2 else 1)] = True
    case = Case(n + ctx, [ctx], [n], hkv, g, d, see=[see], gain=0.5)
    out = attend(b, case, **({} if most_ctx is None else dict(max_query_len=n, max_context_len=most_ctx)))
    assert b.device_error() == 0
    want, spread = case.want()
    few = 2.0 ** -16 + 2.0 ** -13 if ctx < 16 else 2.0 ** -9
    S.close(out, want, ROUND * np.abs(want) + few * spread + 1e-30)


def by_element(case):
    """The 64-bit result with non-finite values where the definition has them (every weight is above zero)."""
    k, v, q = S.f64(case.k), S.f64(case.v), S.f64(case.q)
    clean = np.where(np.isfinite(v), v, 0.0)
    bad = np.where(np.isfinite(v), 0.0, v)
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    for s, (n, length) in enumerate(zip(case.ns, case.lens)):
        see = np.ones((n, length), bool)
        see[:, length - n:] = case.see[s]
        r = slice(case.start[s], case.start[s + 1])
        kk, vv, bb = (S.gather(c, case.tables[s], length, case.nb) for c in (k, clean, bad))
        out[r], spread[r] = S.attend(q[r], kk, vv, case.scale, see)
        g = q.shape[1] // vv.shape[1]
        for i in range(n):
            with np.errstate(invalid="ignore"):
                out[r.start + i] += np.repeat(bb[see[i]].sum(0), g, axis=0)
    return out, spread


@pytest.mark.parametrize("ctx,ns", [([30, 100], [9, 20]), ([0, 700], [130, 17]), ([5000, 3], [16, 150]), ([9], [700])])
@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (1, 1, 64), (2, 8, 64)])
def test_non_finite_values_stay_in_their_element(ctx, ns, hkv, g, d):
    b = S.lib()
    rng = np.random.default_rng(sum(ctx) + sum(ns) + d)
    case = Case(sum(ns), ctx, ns, hkv, g, d)
    for s, n in enumerate(ns):
        base = case.lens[s] - n
        spots = [(int(rng.integers(n)), int(rng.integers(hkv)), int(rng.integers(d)), x)
                 for x in (np.inf, -np.inf, np.nan, np.inf, -np.inf)]
        spots += [(0, 0, d - 1, np.inf), (n - 1, hkv - 1, 0, -np.inf), (n - 1, hkv - 1, 1, np.inf)]
        if n > 1:                                # two signs in one element: NaN for who sees both
            spots += [(0, 0, 5, np.inf), (1, 0, 5, -np.inf)]
        if ctx[s] > 2:                           # a context token's infinity reaches every row
            spots += [(-1, hkv - 1, 11, np.inf)]
        for j, h, e, x in spots:
            pos = base + j
            case.v[case.tables[s, pos // 16], h, pos % 16, e] = x
    out = attend(b, case)
    assert b.device_error() == 0
    got = S.f64(out)
    want, spread = by_element(case)
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    S.close(got[finite], want[finite], (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * spread)[finite])
