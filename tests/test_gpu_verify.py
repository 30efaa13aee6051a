"""verify_drafts against its definition in 64 bits: which rows are kept and
which token follows are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests import verify_helpers as V

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(1)




def outputs(seqs, most):
    return (torch.full((seqs, most), 77, dtype=torch.int32, device="cuda"),
            torch.full((seqs,), 77, dtype=torch.int32, device="cuda"),
            torch.full((seqs,), 77, dtype=torch.int64, device="cuda"))


def check(args, most, max_query_len=None, **kw):
    start, parents, tokens, target, draft, u, final = args
    out = outputs(len(start) - 1, most)
    S.lib().verify_drafts(*out, tokens, parents, start, target, u, final, draft_probs=draft,
                          max_query_len=max_query_len, **kw)
    want = V.walk_all(start, parents, tokens, target, draft, u, final, most)
    for got, ref, what in zip(out, want, ("accepted", "num_accepted", "next_tokens")):
        assert np.array_equal(got.cpu().numpy(), ref), what
    return want


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 100, 1031, 4096, 32003])
def test_trees_of_every_size(vocab, dtype, with_draft):
    ns = [9, 1, 0, 4, 17, 2, 40, 0]
    want = check(V.trees(vocab, ns, vocab, with_draft, dtype), 12)
    assert not with_draft or vocab < 3 or want[1].max() > 1     # (sampled drafts: some stand)


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("seqs", [1, 3, 19, 77, 200, 400])
def test_clusters_of_every_width(seqs, with_draft):
    """Fewer sequences are taken by more CTAs each (eight to one here)."""
    rng = np.random.default_rng(seqs)
    check(V.trees(seqs, list(rng.integers(0, 7, seqs)), 20011 if seqs < 100 else 5003, with_draft), 8)


@pytest.mark.parametrize("with_draft", [True, False])
def test_long_chains_and_wide_trees(with_draft):
    B = S.lib()
    chain = V.trees(5, [300, 1024], 64, with_draft, back=1, sharp=0.3)
    check(chain, 1024)
    check(V.trees(6, [1024, 700], 50, with_draft, back=1000, sharp=0.5), B.MAX_ACCEPTED)


@pytest.mark.parametrize("with_draft", [True, False])
def test_rows_apart_and_unaligned(with_draft):
    start, parents, tokens, target, draft, u, final = V.trees(7, [6, 5, 9], 1001, with_draft)
    wide = torch.full((20, 1013), float("nan"), device="cuda")
    wide[:, 3:1004] = target
    other = None
    if with_draft:
        other = torch.full((20, 2002), float("nan"), device="cuda")
        other[:, :1001] = draft
        other = other[:, :1001]
    check((start, parents, tokens, wide[:, 3:1004], other, u, final), 9)


def dyadic(rows, draft=None):
    """One sequence whose numbers are exact: rows of probabilities in sixteenths."""
    t = torch.tensor(rows, dtype=torch.float32, device="cuda") / 16
    return t, None if draft is None else torch.tensor(draft, dtype=torch.float32, device="cuda") / 16


def one(tokens, parents, target, draft, u, final, most=4):
    t = lambda a, dt: torch.tensor(a, dtype=dt, device="cuda")
    want = check((t([0, len(tokens)], torch.int32), t(parents, torch.int32), t(tokens, torch.int64), target, draft,
                  t(u, torch.float32), t([final], torch.float32)), most)
    return list(want[0][0][:want[1][0]]), int(want[2][0])


def test_borders_are_strict():
    """u q Z < r and running sum > u Z, at equality, with numbers that are exact in every format."""
    p, q = dyadic([[4, 4, 0, 8], [0, 16, 0, 0]], [[8, 4, 4, 0], [16, 0, 0, 0]])
    assert one([0, 0], [-1, 0], p, q, [0, 0.5], 0.0) == ([0], 3)            # 0.5 * 8 = 4: refused; residual 0 0 0 8
    assert one([0, 0], [-1, 0], p, q, [0, 0.5 - 2 ** -25], 0.0) == ([0, 1], 1)
    assert one([0, 0], [-1, 0], p, None, [0, 0.25], 0.0) == ([0], 1)        # certain drafts: 0.25 = p
    assert one([0, 0], [-1, 0], p, None, [0, 0.25 - 2 ** -26], 0.0) == ([0, 1], 1)
    for final, token in ((0.0, 0), (0.25 - 2 ** -26, 0), (0.25, 1), (0.5 - 2 ** -25, 1), (0.5, 3), (1 - 2 ** -24, 3)):
        assert one([5], [-1], p[:1], None, [0], final) == ([0], token)
    # siblings: 0 is refused and leaves [4, 0, 8] of 12, where 1 stands below a third
    p, _ = dyadic([[4, 4, 0, 8]] * 3)
    third = np.nextafter(np.float32(1 / 3), np.float32(0))
    assert one([0, 0, 1], [-1, 0, 0], p, None, [0, 0.9, third], 0.0)[0] == [0, 2]
    assert one([0, 0, 1], [-1, 0, 0], p, None, [0, 0.9, 0.34], 0.7) == ([0], 3)


def test_the_same_token_twice():
    """A refused certain draft proposed again never stands, and is taken off once."""
    p, _ = dyadic([[8, 4, 4, 0]] * 4)
    assert one([0, 0, 0, 0], [-1, 0, 0, 0], p, None, [0, 0.6, 0.0, 0.0], 0.75) == ([0], 2)
    q = dyadic([[8, 4, 4, 0]], [[4, 8, 2, 2]] * 4)[1]
    one([0, 1, 1, 0], [-1, 0, 0, 0], p, q, [0, 0.6, 0.01, 0.2], 0.75)


def test_where_nothing_is_left():
    """Draft and target alike: what was there stands; a row without a positive probability gives no token."""
    p, q = dyadic([[8, 8, 0, 0]] * 3, [[8, 8, 0, 0]] * 3)
    assert one([0, 2, 0], [-1, 0, 0], p, q, [0, 0.5, 1.0], 0.75) == ([0], 1)
    certain, _ = dyadic([[16, 0, 0, 0]] * 3)
    assert one([0, 0, 1], [-1, 0, 0], certain, None, [0, 1.0, 0.0], 0.5) == ([0], 0)
    nothing = torch.full((2, 4), float("nan"), device="cuda")
    nothing[1] = -1.0
    assert one([0], [-1], nothing[:1], None, [0], 0.5) == ([0], -1)
    assert one([0, 1], [-1, 0], nothing, None, [0, 0.0], 0.5) == ([0], -1)


def test_infinitely_many_nans_do_not_spread():
    start, parents, tokens, target, draft, u, final = V.trees(8, [5, 5], 333, True)
    target[:, ::7] = float("nan")
    draft[:, ::5] = float("nan")
    target[:, 1::7] = -target[:, 1::7]
    check((start, parents, tokens, target, draft, u, final), 5)


@pytest.mark.parametrize("most", [1, 2, 3])
def test_as_many_rows_as_there_is_room_for(most):
    """Where max_accepted rows stand the token follows the last of them, whatever hangs below."""
    start, parents, tokens, target, draft, u, final = V.trees(9, [8] * 20, 50, True, back=1, sharp=0.5)
    want = check((start, parents, tokens, target, draft, u * 0.2, final), most)
    assert (want[1] == most).any()


def test_bad_rows_are_flagged_and_passed_over():
    B = S.lib()
    B.device_error()
    start, parents, tokens, target, draft, u, final = V.trees(10, [6, 6, 6], 40, True)
    parents[2], parents[8], tokens[13], tokens[15] = 5, -1, 40, -3
    known = parents.clone()
    known[2] = -7                                # (a later parent is never stood at when its child is tried)
    out = outputs(3, 6)
    B.verify_drafts(*out, tokens, parents, start, target, u, final, draft_probs=draft)
    want = V.walk_all(start, known, tokens, target, draft, u, final, 6)
    for got, ref in zip(out, want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert B.device_error() == B.DEVERR_INDEX
    # row counts that do not fit: below zero, above the bound, past the rows
    for bad, most in (([0, 6, 4, 18], 6), ([0, 6, 12, 18], 5), ([0, 6, 12, 19], 7), ([-1, 4, 8, 12], 6)):
        out = outputs(3, 6)
        B.verify_drafts(*out, tokens, known.clamp(min=0), torch.tensor(bad, dtype=torch.int32, device="cuda"), target, u,
                        final, draft_probs=draft, max_query_len=most)
        for s in range(3):
            n = bad[s + 1] - bad[s]
            if n < 0 or n > most or bad[s] < 0 or bad[s + 1] > 18:
                assert out[1][s] == 0 and out[2][s] == -1 and (out[0][s] == -1).all()
            else:
                assert out[1][s] > 0
        assert B.device_error() & B.DEVERR_LENGTH


def test_tokens_are_distributed_as_the_targets():
    """The token behind row 0, kept draft or next token, has the target's distribution whatever the drafts' is: counts
    of 60000 sequences within 5 standard deviations of their expectation (a wrong one in 2 million such counts)."""
    seqs, vocab = 60000, 8
    rng = np.random.default_rng(11)
    for with_draft in (True, False):
        p = rng.dirichlet(np.ones(vocab) * 0.7)
        q = rng.dirichlet(np.ones(vocab) * 0.7)
        rows = np.tile(p, (4 * seqs, 1))
        tokens = rng.choice(vocab, size=(seqs, 4), p=q)
        if not with_draft:
            tokens[:] = [0, 3, 1, 3]
        t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
        out = outputs(seqs, 4)
        S.lib().verify_drafts(*out, t(tokens.reshape(-1), torch.int64), t(np.tile([-1, 0, 0, 0], seqs), torch.int32),
                              t(np.arange(seqs + 1) * 4, torch.int32), t(rows, torch.float32),
                              t(rng.random(4 * seqs), torch.float32).clamp(max=1 - 2 ** -24),
                              t(rng.random(seqs), torch.float32).clamp(max=1 - 2 ** -24),
                              draft_probs=t(np.tile(q, (4 * seqs, 1)), torch.float32) if with_draft else None)
        kept, follow = out[0][:, 1].cpu().numpy(), out[2].cpu().numpy()
        first = np.where(out[1].cpu().numpy() > 1, tokens[np.arange(seqs), np.maximum(kept, 0)], follow)
        counts = np.bincount(first, minlength=vocab)
        assert np.all(np.abs(counts - seqs * p) <= 5 * np.sqrt(seqs * p * (1 - p)) + 1)


def test_captured_and_on_another_stream():
    B = S.lib()
    args = V.trees(12, [9, 5, 7, 3], 7001, True)
    start, parents, tokens, target, draft, u, final = args
    out = outputs(4, 9)
    call = lambda **kw: B.verify_drafts(*out, tokens, parents, start, target, u, final, draft_probs=draft,
                                        max_query_len=9, **kw)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (13, 14):
        for dst, src in zip(args, V.trees(seed, [9, 5, 7, 3], 7001, True)):
            dst.copy_(src)
        graph.replay()
        want = V.walk_all(*(args[i] for i in (0, 1, 2, 3, 4, 5, 6)), 9)
        assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(out, want))
    side = torch.cuda.Stream()
    for t in out:
        t.fill_(77)
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(out, want))
