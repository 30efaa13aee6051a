"""paged_prefill_attention_scored against the formula in 64 bits: capped
scores, a bias by distance, a window and a prefix seen from both sides, over
poisoned caches."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)


BF = torch.bfloat16
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make(seed, lens, ns, hq, hkv, d, window=0, q_gain=1.0, spare=3):
    """Caches whose rows before what a sequence's first row sees are poisoned; queries with rows behind the last one."""
    first = [max(0, n - m - window + 1) if window else 0 for n, m in zip(lens, ns)]
    k, v, tables, kr, vr = H.paged(seed, lens, hkv, d, BF, first_seen=first)
    rng = np.random.default_rng(seed + 1)
    q = torch.from_numpy((rng.standard_normal((sum(ns) + spare, hq, d)) * q_gain).astype(np.float32)).to(BF).cuda()
    start = np.concatenate([[0], np.cumsum(ns)])
    return q, k, v, tables, kr, vr, start


def compare(out, q, kr, vr, lens, ns, start, scale, cap=0.0, slopes=None, window=0, prefix=None, sequences=None):
    got, qf = S.f64(out), S.f64(q)
    for s in range(len(lens)) if sequences is None else sequences:
        rows = slice(start[s], start[s + 1])
        want, bound = H.attend(qf[rows], kr[s], vr[s], scale, np.arange(lens[s] - ns[s], lens[s]), cap, slopes, window,
                               0 if prefix is None else prefix[s])
        S.close(got[rows], want, bound, f"sequence {s}: {ns[s]} of {lens[s]}")


def run(seed, lens, ns, hq, hkv, d, cap=0.0, slopes=None, window=0, prefix=None, scale=None, q_gain=1.0, **kw):
    B = S.lib()
    B.device_error()
    q, k, v, tables, kr, vr, start = make(seed, lens, ns, hq, hkv, d, window, q_gain)
    out = torch.full_like(q, 55.0)
    scale = d ** -0.5 if scale is None else scale
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32(start), scale, softcap=cap, window=window,
                                     slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                                     prefix_lens=None if prefix is None else i32(prefix), **kw)
    compare(out, q, kr, vr, lens, ns, start, scale, cap, slopes, window, prefix)
    assert (out[start[-1]:] == 55.0).all()           # rows behind the last sequence
    assert B.device_error() == 0


WHOLE = [1, 17, 64, 128, 129, 300, 0, 515]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 4), (6, 2), (16, 4), (8, 1), (16, 1), (64, 1)])
@pytest.mark.parametrize("cap,window,bias,prefix", [(30.0, 0, False, False), (0.0, 70, False, False), (0.0, 0, True, False),
                                                    (0.0, 0, False, True), (8.0, 150, True, True)])
def test_whole_prompts(d, hq, hkv, cap, window, bias, prefix):
    pre = [0, 9, 64, 100, 129, 200, 0, 300] if prefix else None
    run(d + hq, WHOLE, WHOLE, hq, hkv, d, cap, H.alibi(hq) if bias else None, window, pre, q_gain=4.0)


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (24, 2, 64)])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 128, 129, 333, 5000])
def test_chunks_behind_a_context(hq, hkv, d, window):
    lens, ns = [1000, 513, 400, 90, 2049, 129], [1, 200, 130, 0, 77, 128]
    run(window, lens, ns, hq, hkv, d, 0.0, None, window)
    run(window + 1, lens, ns, hq, hkv, d, 20.0, H.alibi(hq), window, prefix=[1000, 350, 390, 1 << 20, 100, 64], q_gain=3.0)


@pytest.mark.parametrize("window", list(range(1, 20)) + [31, 47, 63, 65, 100, 127, 128, 130, 255, 256, 257])
def test_window_edges(window):
    """Every place of the window's start in a block and a chunk; tiles whose chunks do not overlap."""
    lens = [257, 300, 385, 511, 512, 640]
    run(window, lens, lens, 2, 2, 64, 0.0, None, window)
    run(window, lens, [256, 3, 129, 1, 300, 512], 8, 1, 64, 10.0, None, window, q_gain=3.0)


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 200, 255, 256, 300])
def test_prefix_edges(prefix):
    lens = [300, 257, 128, 40]
    run(prefix, lens, lens, 2, 2, 64, prefix=[min(prefix, n) for n in lens])
    run(prefix, lens, [100, 257, 27, 40], 4, 1, 128, prefix=[prefix] * 4, window=90, slopes=H.alibi(4))


@pytest.mark.parametrize("cap", [1e-3, 0.5, 4.0, 20.0, 1e4, 1e15])
def test_caps_of_every_size(cap):
    """Scores far above the cap, around it, where the polynomial ends, and far below."""
    for gain in (0.05, 1.0, 12.0):
        run(3, [140, 700], [140, 300], 8, 2, 128, cap, q_gain=gain)


def test_slopes_of_every_kind():
    slopes = np.array([8.0, 0.5, 0.0, -0.01, 1e-4, -2.0, 100.0, 0.03], dtype=np.float32)
    run(5, [300, 1000, 3], [300, 130, 3], 8, 2, 64, slopes=slopes)
    run(6, [300, 1000, 3], [300, 130, 3], 8, 8, 128, cap=7.0, slopes=slopes, scale=-0.2, window=150, prefix=[80, 900, 2])


@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_scales(scale):
    run(7, [200, 700], [200, 140], 4, 2, 64, scale=scale)
    run(8, [200, 700], [200, 140], 4, 2, 64, cap=3.0, scale=scale, q_gain=5.0)


def test_many_sequences_and_long_contexts():
    rng = np.random.default_rng(9)
    ns = list(rng.integers(0, 40, 150))
    run(9, [int(n + rng.integers(0, 60)) for n in ns], ns, 4, 2, 64, 20.0, window=33)
    run(10, [9000], [140], 4, 1, 128, 30.0, H.alibi(4) * 0.01, q_gain=3.0)
    run(11, [9000, 8000], [1, 260], 4, 1, 64, 30.0, None, 4000, q_gain=3.0)


def test_without_a_transformation_as_plain_prefill():
    """The two kernels round some weights differently: within both bounds of each other."""
    B = S.lib()
    lens, ns = [300, 700, 128], [300, 200, 128]
    q, k, v, tables, kr, vr, start = make(12, lens, ns, 8, 2, 128, spare=0)
    a = B.paged_prefill_attention_scored(torch.empty_like(q), q, k, v, tables, i32(lens), i32(start), 0.088)
    b = B.paged_prefill_attention(torch.empty_like(q), q, k, v, tables, i32(lens), i32(start), 0.088)
    for x in (a, b):
        compare(x, q, kr, vr, lens, ns, start, 0.088)


def test_what_is_not_finite_shows_where_it_is_seen_only():
    """Infinite and NaN keys and values at single positions: rows that do not see them keep their outputs, rows that
    do get what the formula says (NaN for a key; the infinity in its element for a value)."""
    B = S.lib()
    for window, pre, slopes in ((0, 0, None), (90, 0, None), (100, 170, H.alibi(4))):
        lens, ns = [400, 333], [400, 150]
        q, k, v, tables, kr, vr, start = make(13, lens, ns, 4, 2, 64, window)
        bad = {0: {20: float("inf"), 130: float("nan"), 260: -float("inf"), 399: float("inf")}, 1: {200: float("nan"), 300: float("inf")}}
        tb = tables.cpu().numpy()
        for s, at in bad.items():
            for t, x in at.items():
                v[tb[s, t // 16], 1, t % 16, t % 64] = x
        for t in (60, 320):                               # keys of head 0
            k[tb[0, t // 16], 0, t % 16, 5] = float("nan")
        out = torch.empty_like(q)
        B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32(start), 0.125, window=window,
                                         slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                                         prefix_lens=i32([pre, pre]))
        got, qf = S.f64(out), S.f64(q)
        for s in range(2):
            pos = np.arange(lens[s] - ns[s], lens[s])
            see = H.visible(pos, lens[s], window, pre)
            want, bound = H.attend(qf[start[s]:start[s + 1]], kr[s], vr[s], 0.125, pos, 0.0, slopes, window, pre)
            rows = got[start[s]:start[s + 1]]
            mark = np.zeros(rows.shape)                   # what the rows that see something not finite get there
            for t, x in bad[s].items():
                for h in (2, 3):
                    e = see[:, t]
                    was = mark[e, h, t % 64]
                    mark[e, h, t % 64] = np.where(was == 0, x, was + x)
            if s == 0:
                for t in (60, 320):
                    mark[see[:, t], 0:2] = float("nan")
            fine = mark == 0
            assert np.all(np.abs(rows - want)[fine] <= bound[fine]), (window, s)
            assert np.array_equal(np.isnan(rows[~fine]), np.isnan(mark[~fine]))
            inf = np.isinf(mark)
            assert np.array_equal(rows[inf], mark[inf])


def test_bad_pages_lengths_and_prefixes():
    B = S.lib()
    B.device_error()
    lens, ns = [200, 200, 100], [100, 200, 50]
    q, k, v, tables, kr, vr, start = make(14, lens, ns, 4, 2, 64, window=60)
    tables[0, 10] = 1 << 20
    out = torch.full_like(q, 55.0)
    args = (q, k, v, tables)
    B.paged_prefill_attention_scored(out, *args, i32(lens), i32(start), 0.125, window=60)
    kr[0][160:176] = vr[0][160:176] = 0.0
    compare(out, q, kr, vr, lens, ns, start, 0.125, window=60)
    assert B.device_error() == B.DEVERR_BLOCK_ID
    out.fill_(55.0)
    B.paged_prefill_attention_scored(out, *args, i32(lens), i32(start), 0.125, window=60, prefix_lens=i32([-3, 0, 0]))
    compare(out, q, kr, vr, lens, ns, start, 0.125, window=60)
    assert B.device_error() & B.DEVERR_LENGTH
    # more rows than the bound, than the context, than there are; fewer than none
    for starts, kw in (([0, 100, 300, 350], dict(max_query_len=150)), ([0, 100, 301, 350], {}), ([0, 100, 90, 140], {}),
                       ([0, 100, 300, 400], dict(max_query_len=200))):
        out.fill_(55.0)
        B.paged_prefill_attention_scored(out, *args, i32(lens), i32(starts), 0.125, window=60, **kw)
        for s in range(3):
            n, rows = starts[s + 1] - starts[s], slice(starts[s], starts[s + 1])
            if n < 0:
                continue
            if n > lens[s] or n > kw.get("max_query_len", 1 << 30) or starts[s + 1] > q.shape[0]:
                others = [r for z in range(3) if z != s for r in range(starts[z], starts[z + 1])]
                mine = [r for r in range(starts[s], min(starts[s + 1], q.shape[0])) if r not in others]
                assert (out[mine] == 55.0).all()
        assert B.device_error() & B.DEVERR_LENGTH


def test_captured_and_on_another_stream():
    B = S.lib()
    lens, ns = [300, 77], [200, 77]
    q, k, v, tables, kr, vr, start = make(15, lens, ns, 4, 2, 64)
    out, lt, st, pre = torch.empty_like(q), i32(lens), i32(start), i32([250, 30])
    slopes = torch.from_numpy(H.alibi(4)).cuda()
    call = lambda **kw: B.paged_prefill_attention_scored(out, q, k, v, tables, lt, st, 0.125, softcap=8.0, window=90,
                                                         slopes=slopes, prefix_lens=pre, max_query_len=200,
                                                         max_context_len=300, **kw)
    check = lambda: compare(out, q, kr, vr, lens, ns, start, 0.125, 8.0, H.alibi(4), 90, [250, 30])
    call()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        q.copy_(torch.randn_like(q))
        graph.replay()
        check()
    side = torch.cuda.Stream()
    q.copy_(torch.randn_like(q))
    out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    check()
