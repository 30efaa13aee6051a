"""paged_prefill_attention_scored where few query tiles share their keys among
a cluster's CTAs: batches of few rows behind long contexts, with sequences that
leave some of the CTAs nothing."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_gpu_scored_prefill import i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)


# (pairs of tiles times heads: up to about 15 in clusters of eight, 36 of four, 76 of two, on 152 multiprocessors)
SHAPES = [([3000], [9], 4, 1), ([3000, 5, 130], [2, 5, 1], 8, 2), ([2500, 1, 0, 1999], [1, 1, 0, 30], 15, 5),
          ([1500, 700, 129, 1030], [64, 3, 128, 65], 32, 8), ([2100, 40, 900], [300, 40, 200], 8, 4),
          ([1300] * 9, [33, 1, 64, 2, 17, 0, 5, 63, 16], 64, 8), ([700, 550], [700, 550], 64, 1)]


@pytest.mark.parametrize("lens,ns,hq,hkv", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_behind_long_contexts(lens, ns, hq, hkv, d):
    run(d, lens, ns, hq, hkv, d, q_gain=3.0)
    run(d + 1, lens, ns, hq, hkv, d, 20.0, q_gain=4.0)
    run(d + 2, lens, ns, hq, hkv, d, 0.0, H.alibi(hq), window=1100)
    run(d + 3, lens, ns, hq, hkv, d, 9.0, H.alibi(hq) * 0.1, window=777, prefix=[n // 2 for n in lens], q_gain=4.0)


@pytest.mark.parametrize("length", list(range(383, 400)) + [511, 512, 513, 640, 1023, 1024, 1025, 1151, 1153])
def test_every_split_of_the_chunks(length):
    run(length, [length, length - 1], [3, 1], 7, 1, 64, 30.0, q_gain=3.0)
    run(length, [length], [length], 8, 8, 128, window=300)


def test_weight_in_one_place():
    """All of a row's weight with keys of a single CTA, far above the others'; scores that all underflow elsewhere."""
    B = S.lib()
    q, k, v, tables, kr, vr, start = make(4, [4000], [6], 4, 1, 128)
    tb = tables.cpu().numpy()
    for row, t in enumerate((0, 700, 1500, 2222, 3333, 3994)):
        kr[0][t, 0] = S.f64(q[row, row % 4]) * 30
        k[tb[0, t // 16], 0, t % 16] = (q[row, row % 4].float() * 30).to(k.dtype)
        kr[0][t, 0] = S.f64(k[tb[0, t // 16], 0, t % 16])
    out = torch.empty_like(q)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32([4000]), i32(start), 0.5)
    want, bound = H.attend(S.f64(q[:6]), kr[0], vr[0], 0.5, np.arange(3994, 4000))
    S.close(out[:6], want, bound)


def test_what_is_not_finite_in_any_part():
    """As the formula has it in rows that see it, whichever CTA had it; other rows keep their outputs."""
    B = S.lib()
    n, m = 2000, 150
    for window, slopes in ((0, None), (1200, H.alibi(8))):
        q, k, v, tables, kr, vr, start = make(6, [n], [m], 8, 2, 64, window)
        tb = tables.cpu().numpy()
        bad = {900: float("inf"), 1300: float("nan"), 1870: float("inf"), 1951: -float("inf"), 1999: float("nan")}
        for t, x in bad.items():
            v[tb[0, t // 16], 1, t % 16, t % 64] = x
        k[tb[0, 1960 // 16], 0, 1960 % 16, 3] = float("nan")
        out = torch.empty_like(q)
        B.paged_prefill_attention_scored(out, q, k, v, tables, i32([n]), i32(start), 0.125, window=window, slopes=None if slopes is None
                                         else torch.from_numpy(slopes).cuda())
        kr[0][1960, 0] = 0.0
        want, bound = H.attend(S.f64(q[:m]), kr[0], vr[0], 0.125, np.arange(n - m, n), 0.0, slopes, window)
        see = H.visible(np.arange(n - m, n), n, window)
        got = S.f64(out[:m])
        assert np.isnan(got[see[:, 1960], :4]).all()
        got[see[:, 1960], :4] = want[see[:, 1960], :4]
        for c in {t % 64 for t in bad}:
            extra = sum(np.where(see[:, t], x, 0.0) for t, x in bad.items() if t % 64 == c)
            for row in np.flatnonzero(~np.isfinite(extra)):
                assert np.array_equal(got[row, 4:, c], np.full(4, extra[row]), equal_nan=True), (row, c)
                got[row, 4:, c] = want[row, 4:, c]
        S.close(got, want, bound)
        assert B.device_error() == 0


def test_captured_repeated_and_on_another_stream():
    B = S.lib()
    lens, ns = [3000, 77], [20, 4]
    q, k, v, tables, kr, vr, start = make(8, lens, ns, 16, 2, 128)
    args = (q, k, v, tables, i32(lens), i32(start), 0.09)
    most = dict(max_query_len=20, max_context_len=3000)
    a, b, c = (torch.zeros_like(q) for _ in range(3))
    B.paged_prefill_attention_scored(a, *args, softcap=15.0, **most)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        B.paged_prefill_attention_scored(b, *args, softcap=15.0, **most)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.paged_prefill_attention_scored(c, *args, softcap=15.0, **most)
    for _ in range(3):
        c.fill_(3.0)
        graph.replay()
        assert torch.equal(a[:24], b[:24]) and torch.equal(a[:24], c[:24])


def test_bad_pages_in_a_joined_batch():
    B = S.lib()
    B.device_error()
    lens, ns = [2000, 1500], [5, 7]
    q, k, v, tables, kr, vr, start = make(9, lens, ns, 8, 2, 64)
    tables[0, 60] = k.shape[0]                       # reads as zeros, and is reported
    out = torch.empty_like(q)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32(start), 0.125)
    kr[0][960:976] = vr[0][960:976] = 0.0
    for s in range(2):
        rows = slice(start[s], start[s + 1])
        want, bound = H.attend(S.f64(q[rows]), kr[s], vr[s], 0.125, np.arange(lens[s] - ns[s], lens[s]))
        S.close(out[rows], want, bound)
    assert B.device_error() != 0 and B.device_error() == 0
    out.fill_(5.0)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32([0, 6, 5]), 0.125, max_query_len=7)
    assert (out[6:] == 5.0).all()
    assert B.device_error() != 0
