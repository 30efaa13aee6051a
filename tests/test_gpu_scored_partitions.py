"""Decode with transformed scores in partitions: rows and partitions on both
sides of where a warp joins a row."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seqs,hq", [(1, 8), (127, 8), (128, 8), (129, 8)])
@pytest.mark.parametrize("most", [2, 4, 5, 32, 33])
def test_joins_of_few_and_many(most, seqs, hq, dtype):
    """Partitions of 16 tokens, contexts of one to ``most`` of them, an empty one among many."""
    B = S.lib()
    B.device_error()
    rng = np.random.default_rng(most + seqs)
    lens = [16 * most - 3] + [int(x) for x in rng.integers(0, 16 * most + 1, seqs - 1)]
    k, v, tables, kr, vr = H.paged(most, lens, 2, 64, dtype)
    q = torch.randn(seqs, hq, 64, device="cuda").to(dtype)
    out = torch.full_like(q, float("nan"))
    slopes = H.alibi(hq)
    B.paged_decode_attention_scored(out, q, k, v, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125,
                                    softcap=20.0, slopes=torch.from_numpy(slopes).cuda(), partition_tokens=16,
                                    max_context_len=16 * most)
    got, qf = S.f64(out), S.f64(q)
    for s, n in enumerate(lens):
        want, bound = H.attend(qf[s:s + 1], kr[s], vr[s], 0.125, [n - 1], 20.0, slopes, dtype=dtype)
        S.close(got[s:s + 1], want, bound, f"sequence {s} of {n}")
    assert B.device_error() == 0
