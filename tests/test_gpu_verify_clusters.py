"""verify_drafts in clusters of eight CTAs with next to nothing to gather: each
CTA's first sum goes to the others as early as it ever does."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests import verify_helpers as V

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("ns", [[1], [1] * 19, [2, 1, 3, 1, 2]])
def test_first_sums_arrive(ns, with_draft):
    start, parents, tokens, target, draft, u, final = V.trees(len(ns), ns, 20011, with_draft, sharp=1.0)
    want = V.walk_all(start, parents, tokens, target, draft, u, final, 4)
    out = (torch.zeros(len(ns), 4, dtype=torch.int32, device="cuda"),
           torch.zeros(len(ns), dtype=torch.int32, device="cuda"), torch.zeros(len(ns), dtype=torch.int64, device="cuda"))
    B = S.lib()
    for _ in range(200):
        for t in out:
            t.fill_(77)
        B.verify_drafts(*out, tokens, parents, start, target, u, final, draft_probs=draft, max_query_len=3)
        for got, ref in zip(out, want):
            assert np.array_equal(got.cpu().numpy(), ref)
