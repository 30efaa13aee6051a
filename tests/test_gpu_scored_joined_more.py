"""paged_prefill_attention_scored where a cluster's CTAs share a pair's keys,
under prefixes that are seen from both sides, steep biases, and in graphs whose
queries change between replays."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests.test_gpu_scored_prefill import compare, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)


# (few pairs of tiles, so that a pair's keys go to eight, four or two CTAs)
SHAPES = [([3000], [40], 4, 1), ([2500, 700, 64], [260, 3, 64], 8, 2), ([1500, 1030], [200, 130], 16, 8)]


@pytest.mark.parametrize("lens,ns,hq,hkv", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("steep", [1.0, 40.0])
def test_prefixes_without_a_window(steep, d, lens, ns, hq, hkv):
    """The last CTA's keys may all lie behind a row, which a bias that falls off with the distance on both sides all but
    hides; a prefix may end among a call's rows, before them, or hold the whole context."""
    slopes = H.alibi(hq) * np.float32(steep)
    for prefix in ([n - m // 2 for n, m in zip(lens, ns)], [n - m - 5 if n > m + 5 else 0 for n, m in zip(lens, ns)], lens):
        run(d, lens, ns, hq, hkv, d, slopes=slopes, prefix=prefix, q_gain=3.0)
        run(d + 1, lens, ns, hq, hkv, d, 20.0, slopes, prefix=prefix, q_gain=4.0)
        run(d + 2, lens, ns, hq, hkv, d, 20.0, prefix=prefix, q_gain=4.0)


@pytest.mark.parametrize("window", [1, 130, 900])
def test_whole_prompts_under_a_prefix(window):
    """Every row is new: rows at the start see keys of the last CTA's run, within the window only."""
    for length in (640, 1153, 2000):
        run(length, [length], [length], 8, 8, 64, window=window, prefix=[length - 3], slopes=H.alibi(8) * 5)
        run(length + 1, [length], [length], 1, 1, 128, 15.0, window=window, prefix=[length // 3])


def test_queries_change_between_replays():
    B = S.lib()
    lens, ns = [3000, 77], [20, 4]
    q, k, v, tables, kr, vr, start = make(8, lens, ns, 16, 2, 128)
    q2 = make(9, lens, ns, 16, 2, 128, q_gain=2.0)[0]
    out = torch.zeros_like(q)
    args = (k, v, tables, i32(lens), i32(start), 0.09)
    most = dict(max_query_len=20, max_context_len=3000, softcap=15.0)
    now = q.clone()
    B.paged_prefill_attention_scored(out, now, *args, **most)
    compare(out, q, kr, vr, lens, ns, start, 0.09, 15.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.paged_prefill_attention_scored(out, now, *args, **most)
    for x in (q2, q, q2 * 0.5):
        now.copy_(x)
        out.fill_(3.0)
        graph.replay()
        compare(out, x, kr, vr, lens, ns, start, 0.09, 15.0)
        assert (out[24:] == 3.0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    now.copy_(q2)
    out.fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    B.paged_prefill_attention_scored(out, now, *args, stream=side, **most)
    side.synchronize()
    compare(out, q2, kr, vr, lens, ns, start, 0.09, 15.0)


def test_two_calls_at_once():
    """On two streams, over one cache: each has its own outputs and no workspace."""
    B = S.lib()
    calls = []
    for seed, cap in ((3, 0.0), (4, 25.0)):
        q, k, v, tables, kr, vr, start = make(seed, [2600], [30], 8, 2, 64)
        calls.append((q, k, v, tables, kr, vr, start, cap, torch.zeros_like(q), torch.cuda.Stream(), i32([2600]), i32(start)))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, k, v, tables, _, _, _, cap, out, st, n, rows in calls:
            B.paged_prefill_attention_scored(out, q, k, v, tables, n, rows, 0.125, softcap=cap, stream=st,
                                             max_query_len=30, max_context_len=2600)
    torch.cuda.synchronize()
    for q, k, v, tables, kr, vr, start, cap, out, *_ in calls:
        compare(out, q, kr, vr, [2600], [30], start, 0.125, cap)
