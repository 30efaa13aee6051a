"""Tree attention where a row's few keys decide the answer: weights of rows that
see few keys keep their remainders wherever the keys lie."""
import numpy as np
import pytest

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
