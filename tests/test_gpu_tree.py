"""Drafted tokens on the GPU: masks from parents, tree attention against a
64-bit softmax, the move of accepted paths, and a whole speculative step."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S

pytestmark = pytest.mark.gpu

# Bound of an output: its bf16 rounding, 2^-8 of the value, plus sum p |v| times 2^-8 for weights rounded to bf16
# for the tensor cores and 2^-12 for the scores (128 terms in fp32, sum |q k| scale below 32 for these inputs).
WEIGHTS = 2.0 ** -8 + 2.0 ** -12


def random_parents(rng, n, far=6):
    return np.array([-1] + [int(rng.integers(max(-1, i - far), i)) for i in range(1, n)][:max(0, n - 1)],
                    dtype=np.int32)[:n]


def mask_bits(parents):
    n = len(parents)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = parents[j]
    return see


def pack(see, words):
    out = np.zeros((see.shape[0], words), dtype=np.uint64)
    for j in range(see.shape[1]):
        out[:, j // 64] |= see[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


@pytest.mark.parametrize("ns", [[1], [5, 0, 3], [64, 63, 65], [130, 1, 0, 200], [1024]])
def test_masks_from_parents(ns):
    b = S.lib()
    rng = np.random.default_rng(sum(ns))
    parents = [random_parents(rng, n, far=n if n > 100 else 6) for n in ns]
    start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    words = (max(ns) + 63) // 64
    got = b.tree_masks(torch.from_numpy(np.concatenate(parents)).cuda(), torch.from_numpy(start).cuda(), max(ns))
    assert b.device_error() == 0
    want = np.concatenate([pack(mask_bits(p), words) for p in parents])
    assert np.array_equal(got.cpu().numpy(), want)


def test_masks_flag_parents_that_come_later():
    b = S.lib()
    parents = torch.tensor([0, 0, 5, -2], dtype=torch.int32, device="cuda")
    got = b.tree_masks(parents, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), 4)
    assert b.device_error() == b.DEVERR_INDEX
    assert got[:, 0].tolist() == [1, 3, 4, 8]
    out = torch.full((4, 1), 9, dtype=torch.int64, device="cuda")
    b.tree_masks(parents, torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda"), 2, out=out)
    assert b.device_error() == b.DEVERR_LENGTH and bool((out == 9).all())


class Case:
    """A batch of trees: ctx[s] committed tokens, then ns[s] drafts; NaN in every slot past the contexts."""

    def __init__(self, seed, ctx, ns, hkv, g, d, see=None, extra_rows=0, gain=1.0):
        rng = np.random.default_rng(seed)
        self.ns, self.lens = ns, [a + n for a, n in zip(ctx, ns)]
        self.scale = d ** -0.5
        self.tables, self.nb = S.layout(rng, self.lens)
        k, v = (rng.standard_normal((self.nb, hkv, 16, d)) for _ in range(2))
        dead = ~S.live_slots(self.tables, self.lens, self.nb)
        k.transpose(0, 2, 1, 3)[dead] = np.nan
        v.transpose(0, 2, 1, 3)[dead] = np.nan
        self.k, self.v = S.bf16(k * gain), S.bf16(v)
        self.start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        rows = int(self.start[-1]) + extra_rows
        self.q = S.bf16(rng.standard_normal((rows, hkv * g, d)))
        self.see = see if see is not None else [mask_bits(random_parents(rng, n)) if n else np.zeros((0, 0), bool)
                                                for n in ns]
        self.words = max(1, (max(ns) + 63) // 64)
        mask = [pack(m, self.words) for m in self.see]
        self.mask = np.concatenate(mask + [np.zeros((extra_rows, self.words), np.int64)])

    def want(self):
        k, v, q = S.f64(self.k), S.f64(self.v), S.f64(self.q)
        out, spread = np.zeros(q.shape), np.zeros(q.shape)
        for s, (n, length) in enumerate(zip(self.ns, self.lens)):
            see = np.ones((n, length), bool)
            see[:, length - n:] = self.see[s]
            r = slice(self.start[s], self.start[s + 1])
            out[r], spread[r] = S.attend(q[r], S.gather(k, self.tables[s], length, self.nb),
                                         S.gather(v, self.tables[s], length, self.nb), self.scale, see)
        return out, spread

    def cuda(self):
        return [t.cuda() for t in (self.q, self.k, self.v, torch.from_numpy(self.tables),
                                   torch.tensor(self.lens, dtype=torch.int32), torch.from_numpy(self.start),
                                   torch.from_numpy(self.mask))]

    def check(self, out, rows=None):
        want, spread = self.want()
        n = rows if rows is not None else int(self.start[-1])
        S.close(out[:n], want[:n], (2.0 ** -8 * np.abs(want) + WEIGHTS * spread)[:n] + 1e-30)


def attend(b, case, **kw):
    q, k, v, t, n, st, m = case.cuda()
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    b.paged_tree_attention(out, q, k, v, t, n, st, m, case.scale, **kw)
    return out


CTX = [0, 1, 15, 16, 40, 113, 128, 300, 0]
NS = [1, 8, 1, 17, 0, 15, 3, 9, 5]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,g", [(1, 1), (3, 1), (2, 2), (1, 3), (2, 4), (1, 7), (2, 8), (1, 16), (1, 64)])
def test_tree_attention(hkv, g, d):
    b = S.lib()
    case = Case(hkv * 7 + g + d, CTX, NS, hkv, g, d)
    out = attend(b, case)
    assert b.device_error() == 0
    case.check(out)


@pytest.mark.parametrize("ctx,ns", [([500], [64]), ([90, 3], [65, 2]), ([0], [130]), ([1000, 20], [200, 100]),
                                    ([37], [1024]), ([0, 0], [1, 0])])
@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (1, 1, 64), (1, 8, 64)])
def test_wide_trees(ctx, ns, hkv, g, d):
    b = S.lib()
    case = Case(sum(ns) + d, ctx, ns, hkv, g, d)
    out = attend(b, case)
    assert b.device_error() == 0
    case.check(out)


@pytest.mark.parametrize("ctx,ns", [([9000], [5]), ([4096, 30000, 10], [16, 7, 33]), ([2047, 2048, 2049], [1, 1, 1])])
@pytest.mark.parametrize("hkv,g,d", [(2, 4, 128), (1, 16, 128), (2, 1, 64)])
def test_long_contexts(ctx, ns, hkv, g, d):
    b = S.lib()
    case = Case(sum(ctx) + d, ctx, ns, hkv, g, d)
    need = b.tree_workspace_bytes(len(ns), hkv * g, hkv, d, max(ns), max(case.lens))
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
    out = attend(b, case, max_query_len=max(ns), max_context_len=max(case.lens), workspace=ws)
    assert b.device_error() == 0
    case.check(out)


def test_many_sequences():
    b = S.lib()
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(0, 400, size=150)]
    ns = [int(x) for x in rng.integers(0, 12, size=150)]
    case = Case(6, ctx, ns, 4, 4, 128)
    out = attend(b, case, max_query_len=64, max_context_len=4096)
    assert b.device_error() == 0
    case.check(out)


@pytest.mark.parametrize("most_ctx", [150, 4096])
def test_more_sequences_than_threads(most_ctx):
    """900 sequences, some without drafts: short contexts as whole units, and the same batch cut."""
    b = S.lib()
    rng = np.random.default_rng(12)
    ctx = [int(x) for x in rng.integers(0, 100, size=900)]
    ns = [int(x) for x in rng.integers(0, 5, size=900)]
    case = Case(13, ctx, ns, 2, 4, 64)
    out = attend(b, case, max_query_len=5, max_context_len=most_ctx)
    assert b.device_error() == 0
    case.check(out)


def test_one_long_context_among_many_short_ones():
    b = S.lib()
    ctx = [5] * 300 + [20000] + [130] * 20
    case = Case(14, ctx, [2] * 300 + [16] + [1] * 20, 2, 8, 64)
    out = attend(b, case)
    assert b.device_error() == 0
    case.check(out)


def test_no_drafts_at_all():
    b = S.lib()
    case = Case(15, [10, 20], [0, 0], 2, 4, 64, extra_rows=3)
    out = attend(b, case, max_query_len=4)
    assert b.device_error() == 0 and bool(torch.isnan(out.float()).all())
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k, v, t, n, st, m = case.cuda()
    b.kv_accept_layers([k], [v], t, n, st, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.zeros_like(new), new)
    assert new.tolist() == [10, 20] and b.device_error() == 0


def test_masks_that_leave_rows_empty_and_rows_behind_the_last():
    """No context and an empty mask: zeros. Bits past the drafts are ignored. Rows behind the last sequence stay."""
    b = S.lib()
    rng = np.random.default_rng(1)
    ns = [6, 4, 3]
    see = [rng.random((n, n)) < 0.4 for n in ns]
    see[0][2], see[1][0], see[2][:] = False, False, False
    case = Case(2, [0, 20, 0], ns, 2, 4, 64, see=see, extra_rows=5)
    case.mask[:, 0] |= np.int64(-1) << np.int64(6)
    case.mask[case.start[1]:case.start[2], 0] |= np.int64(0x30)
    out = attend(b, case)
    assert b.device_error() == 0
    case.check(out)
    assert not out[2].any() and not out[10:13].any() and bool(torch.isnan(out[13:].float()).all())


def test_infinities_and_nan_in_masked_drafts():
    """A draft that a row does not see can hold anything."""
    b = S.lib()
    see = [np.eye(9, dtype=bool), np.tril(np.ones((20, 20), bool))]
    case = Case(3, [30, 100], [9, 20], 2, 4, 128, see=see)
    for s, j, kv, val in ((0, 3, "k", np.nan), (0, 4, "v", np.nan), (0, 5, "v", np.inf), (0, 6, "k", -np.inf),
                          (1, 18, "v", np.nan), (1, 19, "k", np.inf)):
        pos = case.lens[s] - case.ns[s] + j
        getattr(case, kv)[case.tables[s, pos // 16], :, pos % 16, ::3] = val
    out = attend(b, case)
    keep = [r for r in range(29) if r not in (3, 4, 5, 6, 9 + 18, 9 + 19)]
    want, spread = case.want()
    S.close(S.f64(out)[keep], want[keep], (2.0 ** -8 * np.abs(want) + WEIGHTS * spread)[keep])
    # and what does see them is not made up
    assert not bool(torch.isfinite(out[4].float()).all()) and not bool(torch.isfinite(out[5].float()).all())
    assert bool(torch.isnan(out[3].float()).any()) and not bool(torch.isfinite(out[9 + 18].float()).all())


def test_large_scores_and_scales():
    b = S.lib()
    case = Case(9, [200, 33], [7, 12], 2, 4, 64, gain=30.0)
    for scale in (0.125, -0.125, 0.0):
        case.scale = scale
        q, k, v, t, n, st, m = case.cuda()
        out = torch.zeros_like(q)
        b.paged_tree_attention(out, q, k, v, t, n, st, m, scale)
        want, spread = case.want()
        # scores of |x| up to 2^10: their fp32 error, 64 * 2^-24 * 2^10 = 2^-8, moves the weights too
        S.close(out, want, 2.0 ** -8 * np.abs(want) + (WEIGHTS + 2.0 ** -8) * spread)
    assert b.device_error() == 0


def test_bad_blocks_and_row_counts():
    b = S.lib()
    case = Case(21, [100, 50, 40], [4, 6, 5], 2, 4, 64)
    case.tables[0, 2], case.tables[1, 0] = -7, case.nb
    out = attend(b, case)
    assert b.device_error() == b.DEVERR_BLOCK_ID
    case.check(out)
    case = Case(22, [100, 0, 40], [4, 6, 5], 2, 4, 64)
    q, k, v, t, n, st, m = case.cuda()
    n[1] = 5                                                       # more drafts than context
    out = torch.full_like(q, 7.0)
    b.paged_tree_attention(out, q, k, v, t, n, st, m, case.scale, max_query_len=6, max_context_len=104)
    assert b.device_error() == b.DEVERR_LENGTH
    want, spread = case.want()
    keep = [*range(4), *range(10, 15)]
    S.close(S.f64(out)[keep], want[keep], (2.0 ** -8 * np.abs(want) + WEIGHTS * spread)[keep])
    assert bool((out[4:10] == 7).all())


def test_in_graphs_and_on_streams():
    b = S.lib()
    a, c = Case(31, [3000, 40, 700], [8, 3, 0], 2, 4, 128), Case(32, [64, 5000], [20, 9], 1, 8, 64)
    side = torch.cuda.Stream()
    runs = []
    for case, stream in ((a, None), (c, side)):
        args = case.cuda()
        need = b.tree_workspace_bytes(len(case.ns), args[0].shape[1], args[1].shape[1], args[0].shape[2],
                                      max(case.ns), max(case.lens))
        runs.append((case, args, torch.zeros_like(args[0]),
                     dict(max_query_len=max(case.ns), max_context_len=max(case.lens), stream=stream,
                          workspace=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"))))
    torch.cuda.synchronize()
    for case, args, out, kw in runs:
        b.paged_tree_attention(out, *args, case.scale, **kw)
    torch.cuda.synchronize()
    for case, args, out, kw in runs:
        case.check(out)
    case, args, out, kw = runs[0]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.paged_tree_attention(out, *args, case.scale, **kw)
        graphs.append(g)
    args[0].mul_(0.5)
    case.q = args[0].cpu()
    for g in graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        case.check(out)
    assert b.device_error() == 0


# ---- the accepted path ---------------------------------------------------------------
def accept_reference(caches, tables, lens, ns, accepted, count):
    """Moves in numpy copies; new lengths."""
    new = []
    for s, (length, n) in enumerate(zip(lens, ns)):
        base, a = length - n, int(count[s])
        for c in caches:
            rows = [c[tables[s, (base + d) // 16], :, (base + d) % 16].copy() for d in accepted[s, :a]]
            for j, r in enumerate(rows):
                c[tables[s, (base + j) // 16], :, (base + j) % 16] = r
        new.append(base + a)
    return new


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("hkv,d", [(1, 64), (5, 128), (8, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accepted_paths_move(layers, hkv, d, dtype):
    b = S.lib()
    rng = np.random.default_rng(layers + hkv + d)
    ctx, ns = [0, 1, 15, 30, 7, 100, 3], [1, 8, 20, 64, 0, 5, 70]
    lens = [a + n for a, n in zip(ctx, ns)]
    tables, nb = S.layout(rng, lens)
    accepted = np.full((7, 64), -1, dtype=np.int32)
    count = np.zeros(7, dtype=np.int32)
    for s, n in enumerate(ns):                       # any list of drafts: paths, repeats, falling orders
        count[s] = [min(n, 1), 4, 20, 64, 0, 0, 17][s]
        accepted[s, :count[s]] = rng.integers(0, max(1, n), size=count[s])
    accepted[1, :4] = [0, 2, 3, 7]                   # 2 lies where 3 goes
    kcs, vcs = ([torch.randn(nb, hkv, 16, d, device="cuda").to(dtype) for _ in range(layers)] for _ in range(2))
    want = [S.f64(c) for c in kcs + vcs]
    new_want = accept_reference(want, tables, lens, ns, accepted, count)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    new = torch.zeros(7, dtype=torch.int32, device="cuda")
    start = np.concatenate([[0], np.cumsum(ns)])
    b.kv_accept_layers(kcs, vcs, i32(tables), i32(lens), i32(start), i32(accepted), i32(count), new)
    assert b.device_error() == 0
    assert new.tolist() == new_want
    for got, w in zip(kcs + vcs, want):
        assert np.array_equal(S.f64(got), w)


def test_acceptance_flags_what_is_out_of_range():
    b = S.lib()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = torch.randn(4, 2, 16, 64, device="cuda"), torch.randn(4, 2, 16, 64, device="cuda")
    k0, v0 = kc.clone(), vc.clone()
    tables, start = i32([[0], [1], [2], [99]]), i32([0, 4, 8, 20, 24])
    new = i32([0, 0, 0, 0])
    # a draft out of range is left out; a count past the drafts is clamped; more drafts than context moves nothing;
    # a bad block is skipped
    b.kv_accept_layers([kc], [vc], tables, i32([8, 8, 9, 8]), start, i32([[0, 4, 2], [1, 1, 1], [1, 2, 3], [1, 2, 3]]),
                       i32([3, 9, 2, 2]), new)
    assert b.device_error() == b.DEVERR_INDEX | b.DEVERR_LENGTH | b.DEVERR_BLOCK_ID
    assert new.tolist() == [7, 7, 9, 6]
    for c, c0 in ((kc, k0), (vc, v0)):
        want = c0.clone()
        want[0, :, 6] = c0[0, :, 6]
        for j in range(3):
            want[1, :, 4 + j] = c0[1, :, 5]
        assert torch.equal(c, want)


def test_acceptance_without_sequences_layers_or_room():
    b = S.lib()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    new = i32([5])
    b.kv_accept_layers([], [], i32([[0]]), i32([3]), i32([0, 1]), i32([[0]]), i32([1]), new)
    assert new.item() == 5
    c = torch.randn(1, 1, 16, 64, device="cuda")
    b.kv_accept_layers([c], [c.clone()], i32([[0]]), i32([3]), i32([0, 1]), torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                       i32([0]), new)
    assert new.item() == 2 and b.device_error() == 0


def test_acceptance_replayed_from_a_graph():
    """Each replay moves the path of that step: counts, paths and lengths change in place."""
    b = S.lib()
    rng = np.random.default_rng(40)
    ns, ctx = [6, 9], [20, 3]
    lens = [a + n for a, n in zip(ctx, ns)]
    tables, nb = S.layout(rng, lens)
    kc, vc = (torch.randn(nb, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    t, n, st = i32(tables), i32(lens), i32([0, 6, 15])
    acc, count, new = i32([[0, 0, 0], [0, 0, 0]]), i32([0, 0]), i32([0, 0])
    ptrs = b.layer_pointers([kc]), b.layer_pointers([vc])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.kv_accept_layers([kc], [vc], t, n, st, acc, count, new, ptrs=ptrs)
    for paths, counts in (([[0, 2, 5], [1, 3, 8]], [3, 2]), ([[4, 1, 0], [8, 8, 8]], [2, 3])):
        want = [S.f64(kc), S.f64(vc)]
        new_want = accept_reference(want, tables, lens, ns, np.array(paths), counts)
        acc.copy_(i32(paths))
        count.copy_(i32(counts))
        g.replay()
        torch.cuda.synchronize()
        assert new.tolist() == new_want and np.array_equal(S.f64(kc), want[0]) and np.array_equal(S.f64(vc), want[1])
    assert b.device_error() == 0


# ---- a speculative step as a server runs it ---------------------------------------------
def test_a_speculative_step_end_to_end():
    """Drafts normalised, rotated and appended; the tree attended; a path accepted in every layer; the next decode step
    attends the same rows as if the path had been decoded token by token."""
    b = S.lib()
    torch.manual_seed(3)
    rng = np.random.default_rng(3)
    hq, hkv, d, layers = 8, 2, 128, 2
    ctx, ns = [37, 5, 120], [7, 6, 9]
    path = [[0, 2, 5], [0], [1, 4, 6, 8]]
    tables, nb = S.layout(rng, [a + n + 1 for a, n in zip(ctx, ns)])
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    dev = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    slot = lambda s, p: tables[s, p // 16] * 16 + p % 16  # noqa: E731
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    freq = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    parents = [np.array([-1, -1, 0, 0, 1, 2, 4, 3, 6][:n], dtype=np.int32) for n in ns]
    depth = [[0] * n for n in ns]
    for s, p in enumerate(parents):
        for i, up in enumerate(p):
            depth[s][i] = 0 if up < 0 else depth[s][up] + 1
    tree = [torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2 * layers)]
    line = [torch.zeros_like(c) for c in tree]
    outs = {}
    for layer in range(layers):
        kc, vc, lk, lv = tree[layer], tree[layers + layer], line[layer], line[layers + layer]
        # the committed context
        for s, n in enumerate(ctx):
            x = torch.randn(n, hq + 2 * hkv, d, device="cuda").bfloat16()
            q, k, v = x.split([hq, hkv, hkv], 1)
            for a, c in ((kc, vc), (lk, lv)):
                b.qk_norm_rope_append(torch.empty(n, hq, d, dtype=x.dtype, device="cuda"), q, k, v, torch.arange(n, device="cuda"),
                                      freq, dev([slot(s, p) for p in range(n)]).long(), a, c, q_weight=w, k_weight=w)
        # the drafts, at the positions their depths give them
        T = sum(ns)
        x = torch.randn(T, hq + 2 * hkv, d, device="cuda").bfloat16()
        q, k, v = x.split([hq, hkv, hkv], 1)
        pos = [ctx[s] + depth[s][i] for s in range(3) for i in range(ns[s])]
        slots = [slot(s, ctx[s] + i) for s in range(3) for i in range(ns[s])]
        qr = torch.empty(T, hq, d, dtype=x.dtype, device="cuda")
        b.qk_norm_rope_append(qr, q, k, v, dev(pos), freq, dev(slots).long(), kc, vc, q_weight=w, k_weight=w)
        start = i32(np.concatenate([[0], np.cumsum(ns)]))
        lens = i32([a + n for a, n in zip(ctx, ns)])
        mask = b.tree_masks(i32(np.concatenate(parents)), start, max(ns))
        out = torch.empty_like(qr)
        b.paged_tree_attention(out, qr, kc, vc, i32(tables), lens, start, mask, d ** -0.5)
        # the same path, one decode step at a time
        first = np.concatenate([[0], np.cumsum(ns)])
        for j in range(4):
            rows = [(s, first[s] + path[s][j]) for s in range(3) if j < len(path[s])]
            ids = dev([r for _, r in rows]).long()
            lq = torch.empty(len(rows), hq, d, dtype=x.dtype, device="cuda")
            b.qk_norm_rope_append(lq, q[ids], k[ids], v[ids], dev([ctx[s] + j for s, _ in rows]), freq,
                                  dev([slot(s, ctx[s] + j) for s, _ in rows]).long(), lk, lv, q_weight=w, k_weight=w)
            lo = torch.empty_like(lq)
            b.paged_decode_attention(lo, lq, lk, lv, i32(tables[[s for s, _ in rows]]), i32([ctx[s] + j + 1 for s, _ in rows]),
                                     d ** -0.5)
            assert torch.equal(lq, qr[ids])
            # two kernels, each within bf16 rounding of the same value: inputs and outputs are of size 1
            assert float((lo.float() - out[ids].float()).abs().max()) < 2 * (2.0 ** -8 + WEIGHTS) * 4
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    acc = np.zeros((3, 4), dtype=np.int32)
    for s in range(3):
        acc[s, :len(path[s])] = path[s]
    b.kv_accept_layers(tree[:layers], tree[layers:], i32(tables), lens, start, i32(acc), i32([len(p) for p in path]), new)
    assert new.tolist() == [a + len(p) for a, p in zip(ctx, path)]
    for got, want in zip(tree, line):
        for s, n in enumerate(new.tolist()):
            for p in range(n):
                assert torch.equal(got[tables[s, p // 16], :, p % 16], want[tables[s, p // 16], :, p % 16]), (s, p)
    assert b.device_error() == 0


def test_a_quantised_server_end_to_end():
    """A prompt quantised as it is written, read back for prefill, then decode over the tiles: each against a cache of
    the same values in bf16."""
    b = S.lib()
    torch.manual_seed(5)
    rng = np.random.default_rng(5)
    hq, hkv, d = 8, 2, 128
    lens = [45, 16, 3]
    tables, nb = S.layout(rng, [n + 1 for n in lens])
    dev = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    kq, vq = b.e4m3_cache(nb, hkv, d), b.e4m3_cache(nb, hkv, d)
    kb, vb = (torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    T = sum(lens)
    k, v = (torch.randn(T, hkv, d, device="cuda").bfloat16() for _ in range(2))
    slots = dev([tables[s, p // 16] * 16 + p % 16 for s, n in enumerate(lens) for p in range(n)]).long()
    b.kv_append_e4m3(k, v, slots, kq, vq)
    b.dequantize_blocks(kb, vb, kq, vq, dev(np.stack([np.arange(nb)] * 2, 1)))
    q = torch.randn(T, hq, d, device="cuda").bfloat16()
    out = torch.empty_like(q)
    start = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    tab = dev(tables)
    b.paged_prefill_attention(out, q, kb, vb, tab, dev(np.array(lens, dtype=np.int32)), start, d ** -0.5)
    for s, n in enumerate(lens):
        kk, vv = (S.gather(S.tile_values(c), tables[s], n, nb) for c in (kq, vq))
        r = slice(int(start[s]), int(start[s + 1]))
        want, spread = S.attend(S.f64(q[r]), kk, vv, d ** -0.5, np.tril(np.ones((n, n), bool)))
        S.close(out[r], want, 2.0 ** -8 * np.abs(want) + WEIGHTS * spread)
    # the next token, its key turned, through the fused pass into the tiles
    x = torch.randn(3, hq + 2 * hkv, d, device="cuda").bfloat16()
    qn, kn, vn = x.split([hq, hkv, hkv], 1)
    qr = torch.empty(3, hq, d, dtype=x.dtype, device="cuda")
    freq = torch.rand(64, device="cuda")
    b.qk_norm_rope_append(qr, qn, kn, vn, dev(np.array(lens)), freq,
                          dev([tables[s, n // 16] * 16 + n % 16 for s, n in enumerate(lens)]).long(), kq, vq)
    od = torch.empty_like(qr)
    b.paged_decode_attention_e4m3(od, qr, kq, vq, tab, dev(np.array([n + 1 for n in lens], dtype=np.int32)), d ** -0.5)
    for s, n in enumerate(lens):
        kk, vv = (S.gather(S.tile_values(c), tables[s], n + 1, nb) for c in (kq, vq))
        want, spread = S.attend(S.f64(qr[s:s + 1]), kk, vv, d ** -0.5)
        S.close(od[s:s + 1], want, 2.0 ** -8 * np.abs(want) + WEIGHTS * spread)
    assert b.device_error() == 0
