"""Decode over e4m3 tiles where the rows' scale bytes say little about their
size: blocks that nothing was written to. Against a 64-bit softmax over the
values that the tiles stand for, under the bound of the ordinary decode tests."""
import pytest
import torch

from tests import serving_helpers as S
from tests.test_gpu_e4m3 import Case

pytestmark = pytest.mark.gpu


def decode(b, c, dtype=torch.float32, **kw):
    q, k, v, t, n = c.cuda()
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    b.paged_decode_attention_e4m3(out, q, k, v, t, n, c.scale, **kw)
    return out


def freshen(c, s, blocks):
    """Blocks of sequence s as e4m3_cache makes them: zero codes, zero scale bytes."""
    for j in blocks:
        c.k[c.tables[s, j]] = 0
        c.v[c.tables[s, j]] = 0


@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (1, 1, 64), (1, 16, 128), (2, 9, 64)])
def test_blocks_that_nothing_was_written_to(hkv, g, d):
    """A fresh block's rows are zeros, as in any other cache: they share the weight and add nothing."""
    b = S.lib()
    c = Case(50 + d + g, [48, 100, 16, 70, 250], hkv, g, d)
    freshen(c, 0, [0])              # before a written block
    freshen(c, 1, [2, 3, 6])        # between, and at the ragged end
    freshen(c, 2, [0])              # nothing else
    freshen(c, 3, [3])
    for dtype in (torch.float32, torch.bfloat16):
        out = decode(b, c, dtype)
        assert b.device_error() == 0
        c.check(out)


@pytest.mark.parametrize("hkv,g,d", [(1, 4, 128), (2, 8, 64), (1, 16, 128)])
def test_fresh_blocks_that_fill_whole_segments(hkv, g, d):
    """One long context is cut among the workers: some of them see fresh blocks only."""
    b = S.lib()
    c = Case(60 + d + g, [20000, 400], hkv, g, d)
    freshen(c, 0, [*range(0, 90), *range(200, 300), *range(1240, 1250)])
    out = decode(b, c)
    assert b.device_error() == 0
    c.check(out)
