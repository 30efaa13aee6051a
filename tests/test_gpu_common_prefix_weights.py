"""Rows that give nearly all of their weight to a few of the first tokens of a
common prefix: those weights have 16 bits, as plain decode's of the first 64
tokens have."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_gpu_common_prefix import i32, make

pytestmark = pytest.mark.gpu


def heavy(seed, lens, shared, hq, hkv, d, tokens):
    """All tokens but those at ``tokens`` lie 21 or 30 below in the exponent (element 0 of q and k)."""
    q, k, v, tables, rows = make(seed, [0, len(lens)], lens, [shared], hq, hkv, d, 0.3)
    q[..., 0] = 8.0
    k[..., 0] = torch.where(torch.isfinite(k[..., 0]), -30.0, k[..., 0])
    tb = tables.cpu().numpy()
    for t in tokens:
        k[tb[0, t // 16], :, t % 16, 0] = 0.0
    for kr, _ in rows:
        kr[..., 0] = -30.0
        kr[list(tokens), :, 0] = 0.0
    return q, k, v, tables, rows


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,seqs,shared", [(8, 2, 5, 8), (32, 8, 40, 9), (16, 1, 9, 64), (7, 7, 3, 200), (8, 8, 150, 12)])
def test_few_first_tokens_carry_the_weight(hq, hkv, seqs, shared, d):
    """Bound: the output's rounding, 2^-16 of the weights (bf16 and the bf16 of what it leaves: half a step of 2^-8 of half
    a step of 2^-8), once in the product and once in the sum, and the scores' errors."""
    B = S.lib()
    rng = np.random.default_rng(seqs)
    lens = [16 * shared + int(n) for n in rng.integers(0, 90, seqs)]
    q, k, v, tables, rows = heavy(seqs + d, lens, shared, hq, hkv, d, (0, 17, 63))
    scale = d ** -0.5
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    B.paged_decode_attention_common_prefix(outs[0], q, k, v, tables, i32(lens), scale, i32([0, seqs]), i32([shared]))
    B.paged_decode_attention(outs[1], q, k, v, tables, i32(lens), scale)
    for s, n in enumerate(lens):
        want, bound = H.attend(S.f64(q[s:s + 1]), *rows[s], scale, [n - 1], weight_step=2.0 ** -16)
        if hq != hkv:                                   # (plain decode of one head a kv head keeps its weights in fp32)
            S.close(outs[1][s:s + 1], want, bound, f"plain, sequence {s}")
        S.close(outs[0][s:s + 1], want, bound, f"sequence {s}")


@pytest.mark.parametrize("shared", [8, 9, 150])
def test_infinities_and_nans_among_the_first_tokens(shared):
    """Negative remainders of the weights do not turn an infinity into NaN."""
    B = S.lib()
    lens = [16 * shared + 33] * 5
    q, k, v, tables, rows = make(21, [0, 5], lens, [shared], 8, 2, 128)
    tb = tables.cpu().numpy()
    for t in range(0, 128, 3):
        v[tb[0, t // 16], 1, t % 16, t] = float("inf")
    v[tb[0, 6], 1, 5, 1] = float("nan")
    out = torch.empty_like(q)
    B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.09, i32([0, 5]), i32([shared]))
    got = S.f64(out)
    assert np.all(got[:, 4:, 0:128:3] == np.inf) and np.isnan(got[:, 4:, 1]).all()
    for s in range(5):
        want, bound = H.attend(S.f64(q[s:s + 1]), *rows[s], 0.09, [lens[s] - 1])
        for c in (*range(0, 128, 3), 1):
            got[s, 4:, c] = want[0, 4:, c]
        S.close(got[s:s + 1], want, bound)
