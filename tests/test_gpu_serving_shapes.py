"""Shapes that the serving calls refuse although their first sizes fit."""
import pytest
import torch

from tests import serving_helpers as S
from tests.test_gpu_tree import Case

pytestmark = pytest.mark.gpu


def test_lengths_of_two_dimensions_are_refused():
    """[S, 2] lengths would be read as the first S numbers."""
    b = S.lib()
    case = Case(1, [20, 5], [3, 2], 1, 2, 64)
    q, k, v, t, n, st, m = case.cuda()
    two = torch.stack([n, n], 1).contiguous()
    with pytest.raises(ValueError):
        b.paged_tree_attention(torch.zeros_like(q), q, k, v, t, two, st, m, case.scale, max_query_len=3, max_context_len=23)
    accepted = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        b.kv_accept_layers([k], [v], t, two, st, accepted, torch.zeros_like(n), torch.zeros_like(n))
    with pytest.raises(ValueError):
        b.paged_decode_attention_e4m3(q[:2], q[:2], *(b.e4m3_cache(2, 1, 64) for _ in "kv"), t, two, case.scale)
    assert b.device_error() == 0
