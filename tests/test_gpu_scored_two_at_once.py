"""Two calls at once, on two streams with a workspace each, eager and as graphs:
decode with transformed scores, under a common prefix, and verification of
drafts."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests import verify_helpers as V
from tests.test_gpu_common_prefix import compare as compare_common
from tests.test_gpu_common_prefix import make as make_common

pytestmark = pytest.mark.gpu
i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def together(calls, times=15):
    """Each call(stream) over and over on a stream of its own; then the same from two graphs."""
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(times):
        for call, st in zip(calls, streams):
            call(st)
    torch.cuda.synchronize()
    yield "eager"
    graphs = []
    for call, st in zip(calls, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            call(st)
    torch.cuda.synchronize()
    for _ in range(times):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    yield "graphs"


def test_common_prefixes():
    B = S.lib()
    made, calls = [], []
    for seed, seqs, shared, hq, hkv, d in ((1, 40, 60, 8, 2, 128), (2, 70, 25, 8, 8, 64)):
        lens = [16 * shared + 7 * s for s in range(seqs)]
        q, k, v, tables, rows = make_common(seed, [0, seqs // 2, seqs], lens, [shared, shared - 5], hq, hkv, d)
        out = torch.zeros_like(q)
        ws = torch.zeros(B.common_prefix_workspace_bytes(seqs, hq, hkv, d), dtype=torch.uint8, device="cuda")
        args = (out, q, k, v, tables, i32(lens), d ** -0.5, i32([0, seqs // 2, seqs]), i32([shared, shared - 5]))
        kw = dict(max_group_size=seqs, max_context_len=max(lens), workspace=ws)
        calls.append(lambda st, args=args, kw=kw: B.paged_decode_attention_common_prefix(*args, stream=st, **kw))
        made.append((out, q, rows, lens, d ** -0.5))
    for how in together(calls):
        for out, q, rows, lens, scale in made:
            compare_common(out, q, rows, lens, scale, how)
            out.fill_(float("nan"))


@pytest.mark.parametrize("parts", [0, 64, -1])
def test_decode(parts):
    B = S.lib()
    made, calls = [], []
    for seed, cap, window in ((3, 20.0, 0), (4, 0.0, 300)):
        lens = [int(x) for x in np.random.default_rng(seed).integers(1, 900, 50)]
        k, v, tables, kr, vr = H.paged(seed, lens, 2, 64, torch.bfloat16, window)
        q = torch.randn(50, 8, 64, device="cuda").to(torch.bfloat16)
        out = torch.zeros_like(q)
        ws = torch.zeros(B.workspace_bytes(50, 8, 2, 64, max(lens), parts), dtype=torch.uint8, device="cuda")
        args = (out, q, k, v, tables, i32(lens), 0.125)
        kw = dict(softcap=cap, window=window, max_context_len=max(lens), partition_tokens=parts, workspace=ws)
        calls.append(lambda st, args=args, kw=kw: B.paged_decode_attention_scored(*args, stream=st, **kw))
        made.append((out, q, kr, vr, lens, cap, window))
    for how in together(calls):
        for out, q, kr, vr, lens, cap, window in made:
            for s, n in enumerate(lens):
                want, bound = H.attend(S.f64(q[s:s + 1]), kr[s], vr[s], 0.125, [n - 1], cap, None, window)
                S.close(out[s:s + 1], want, bound, f"{how}, sequence {s} of {n}")
            out.fill_(float("nan"))


def test_verification():
    B = S.lib()
    made, calls = [], []
    for seed, ns, vocab, with_draft in ((5, [7] * 30, 9001, True), (6, [3, 9, 1, 5] * 4, 20011, False)):
        args = V.trees(seed, ns, vocab, with_draft)
        start, parents, tokens, target, draft, u, final = args
        out = tuple(torch.zeros(shape, dtype=dt, device="cuda") for shape, dt in
                    (((len(ns), 6), torch.int32), ((len(ns),), torch.int32), ((len(ns),), torch.int64)))
        calls.append(lambda st, out=out, a=args: B.verify_drafts(*out, a[2], a[1], a[0], a[3], a[5], a[6], draft_probs=a[4],
                                                                 max_query_len=9, stream=st))
        made.append((out, V.walk_all(*args, 6)))
    for how in together(calls):
        for out, want in made:
            for got, ref in zip(out, want):
                assert np.array_equal(got.cpu().numpy(), ref), how
                got.fill_(-7)
