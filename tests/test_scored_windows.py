"""Windows past 32 bits see everything (they were cut to their low 32 bits: a
window of 2^32 + 5 was one of 5), and negative ones are refused."""
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S

FAR = [1 << 31, (1 << 32) + 5, 1 << 40]


def test_as_the_abi_takes_them():
    B = S.lib()
    assert [B._window(w) for w in (0, 1, (1 << 31) - 1)] == [0, 1, (1 << 31) - 1]
    assert all(B._window(w) == (1 << 31) - 1 for w in FAR)
    assert all(B._window(-w) == -1 for w in [1, 5] + FAR)


@pytest.mark.gpu
@pytest.mark.parametrize("window", FAR)
def test_far_windows_see_everything(window):
    B = S.lib()
    lens = [70, 300, 1]
    k, v, tables, _, _ = H.paged(1, lens, 2, 64, torch.bfloat16)
    q = torch.randn(3, 8, 64, device="cuda").to(torch.bfloat16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    for call, more in ((B.paged_decode_attention_scored, ()), (B.paged_prefill_attention_scored, (i32([0, 1, 2, 3]),))):
        a, b = torch.zeros_like(q), torch.ones_like(q)
        call(a, q, k, v, tables, i32(lens), *more, 0.125, window=window)
        call(b, q, k, v, tables, i32(lens), *more, 0.125)
        assert torch.equal(a, b)
        for bad in (-1, -window):
            with pytest.raises(B.PagedKVError):
                call(a, q, k, v, tables, i32(lens), *more, 0.125, window=bad)
