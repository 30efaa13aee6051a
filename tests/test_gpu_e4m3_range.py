"""Decode over e4m3 tiles where the rows' scale bytes say little about their
size, or lie far apart: blocks that nothing was written to, value rows of
zeros, blocks with a bad id, one value row far larger than the others; and
contexts around the length from which they are cut among the workers. Each
against a 64-bit softmax over the values that the tiles stand for, under the
bound of the ordinary decode tests."""
import numpy as np
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


def set_value_row(c, s, token, x):
    """Value row `token` of sequence s, every kv head: the row x [D]."""
    codes, scales = S.e4m3_rows(x)
    d = len(x)
    blk, off = c.tables[s, token // 16], token % 16
    c.v[blk, :, off * d:(off + 1) * d] = torch.from_numpy(codes)
    c.v[blk, :, 16 * d + off] = int(scales)


def lift_key(c, s, token, by):
    """Key row `token` of sequence s gives its one query head a score of about `by` (natural log)."""
    q = S.f64(c.q[s, 0])
    codes, scales = S.e4m3_rows(q * (by / c.scale / (q @ q)))
    d = len(q)
    blk, off = c.tables[s, token // 16], token % 16
    c.k[blk, :, off * d:(off + 1) * d] = torch.from_numpy(codes)
    c.k[blk, :, 16 * d + off] = int(scales)


@pytest.mark.parametrize("size", [2.0 ** -7, 2.0 ** -10, 2.0 ** -17, 2.0 ** -40, 1.0, 300.0])
@pytest.mark.parametrize("d", [64, 128])
def test_a_value_row_of_zeros_under_the_highest_score(d, size):
    """It takes most of the weight, adds nothing, and costs the other rows' weights no precision."""
    b = S.lib()
    c = Case(70 + d, [64, 33, 500], 1, 1, d)
    rng = np.random.default_rng(d)
    for s, n in enumerate(c.lens):
        for t in range(n):
            set_value_row(c, s, t, rng.standard_normal(d) * size)
        for t in (5, n - 1):
            set_value_row(c, s, t, np.zeros(d))
            lift_key(c, s, t, 6.0)
    for most in (max(c.lens), 512):
        out = decode(b, c, max_context_len=most)
        assert b.device_error() == 0
        c.check(out)


def test_a_row_of_nan_only_costs_the_others_nothing():
    """A value row whose elements are NaN and zeros: NaN where it is NaN, the others' average elsewhere."""
    b = S.lib()
    d = 128
    c = Case(75, [40], 1, 1, d)
    rng = np.random.default_rng(1)
    for t in range(40):
        set_value_row(c, 0, t, rng.standard_normal(d) * 2.0 ** -17)
    set_value_row(c, 0, 7, np.where(np.arange(d) == 3, np.nan, 0.0))
    lift_key(c, 0, 7, 6.0)
    out = S.f64(decode(b, c))
    assert b.device_error() == 0 and np.isnan(out[0, 0, 3])
    set_value_row(c, 0, 7, np.zeros(d))
    want, spread = c.want()
    rest = np.arange(d) != 3
    S.close(out[..., rest], want[..., rest], (2.0 ** -24 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread)[..., rest])


@pytest.mark.parametrize("size", [2.0 ** -17, 1.0])
def test_a_bad_block_costs_small_values_nothing(size):
    """A block id out of range reads as zeros, beside values of any size."""
    b = S.lib()
    d = 128
    c = Case(80, [90], 1, 1, d)
    rng = np.random.default_rng(2)
    for t in range(90):
        set_value_row(c, 0, t, rng.standard_normal(d) * size)
    c.q *= 4                                     # scores of size 4 around the zeros' 0
    c.tables[0, 2] = c.nb + 5
    out = decode(b, c)
    assert b.device_error() == b.DEVERR_BLOCK_ID
    c.check(out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("far", [12, 20, 24])
def test_one_value_row_far_above_the_others(far, d):
    """An outlier in one element of one row must not round away the other elements' averages: a weight keeps f16's
    11 bits down to 2^-25 of the largest weighted value."""
    b = S.lib()
    c = Case(90 + far, [300, 20], 1, 4, d)
    rng = np.random.default_rng(far)
    for s, n in enumerate(c.lens):
        for t in range(n):
            set_value_row(c, s, t, np.sign(rng.standard_normal(d)) * rng.uniform(1.0, 1.75, d))
        set_value_row(c, s, n // 2, np.where(np.arange(d) == 9, 2.0 ** far, 0.0))
    c.q *= 0.03                                  # weights within a factor of two of one another
    out = decode(b, c)
    assert b.device_error() == 0
    c.check(out)


def test_scores_as_large_as_fp32_resolves():
    """Scores around 2^27, where the step of fp32 exceeds the reference's distance from the maximum: one row takes all
    the weight."""
    b = S.lib()
    d = 64
    c = Case(95, [100, 40], 1, 1, d)
    c.q[:] = 2.0 ** 45
    c.k[:, :, :16 * d] = 0x30                    # 0.5
    c.k[:, :, 16 * d:] = 127 - 20
    c.scale = 2.0 ** -3
    for s, top in ((0, 33), (1, 17)):
        c.k[c.tables[s, top // 16], 0, 16 * d + top % 16] = 127 - 19
    out = S.f64(decode(b, c))
    assert b.device_error() == 0
    values = S.tile_values(c.v)
    for s, top in ((0, 33), (1, 17)):
        want = values[c.tables[s, top // 16], 0, top % 16]
        assert np.all(np.abs(out[s, 0] - want) <= (2.0 ** -11 + 2.0 ** -24) * np.abs(want))


@pytest.mark.parametrize("most", [96, 97, 128, 257])
@pytest.mark.parametrize("hkv,g,d,seqs", [(4, 4, 128, 300), (3, 1, 64, 40), (1, 16, 128, 7), (1, 2, 64, 4100)])
def test_short_contexts_whole_and_cut(hkv, g, d, seqs, most):
    """Contexts on both sides of the length up to which a worker takes whole units."""
    b = S.lib()
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(0, 97 if seqs < 1000 else 20, size=seqs)]
    lens[0], lens[-1] = 96, 0
    c = Case(99, lens, hkv, g, d)
    out = decode(b, c, torch.bfloat16, max_context_len=most)
    assert b.device_error() == 0
    c.check(out)
