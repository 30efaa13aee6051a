"""verify_drafts where its numbers are delicate: drafts tried on probabilities
that are none, comparisons at their border behind refusals, and remainders of
less than a unit of the sums."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import serving_helpers as S
from tests import verify_helpers as V

pytestmark = pytest.mark.gpu


def call(ns, parents, tokens, target, draft, u, final, most=4):
    """Outputs on the host, of numpy inputs; probabilities may be CPU tensors of their type."""
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
    rows = lambda a: None if a is None else a.cuda() if isinstance(a, torch.Tensor) else t(a, torch.float32)
    seqs = len(ns)
    out = (torch.full((seqs, most), 77, dtype=torch.int32, device="cuda"),
           torch.full((seqs,), 77, dtype=torch.int32, device="cuda"),
           torch.full((seqs,), 77, dtype=torch.int64, device="cuda"))
    S.lib().verify_drafts(*out, t(tokens, torch.int64), t(parents, torch.int32),
                          t(np.concatenate([[0], np.cumsum(ns)]), torch.int32), rows(target), t(u, torch.float32),
                          t(final, torch.float32), draft_probs=rows(draft))
    return [o.cpu().numpy() for o in out]


STRANGE = [float("nan"), -0.5, float("inf"), -float("inf"), 2.0, -0.0, 1.0, 0.25]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seed", range(6))
def test_drafts_are_tried_on_cleaned_probabilities(seed, dtype):
    """Every pair of strange p and q at a drafted token, of a first draft (where nothing was refused) and of a second
    behind one that p gives nothing: negative ones and NaN count as 0, ones above 1 as 1."""
    rng = np.random.default_rng(seed)
    pairs = [(a, b, second) for a in STRANGE + [0.0] for b in STRANGE + [0.0] for second in (False, True)]
    n, vocab = 3, 9
    p = rng.dirichlet(np.ones(vocab), size=len(pairs) * n)
    q = rng.dirichlet(np.ones(vocab), size=len(pairs) * n)
    tokens, parents = np.zeros((len(pairs), n), dtype=np.int64), np.tile([-1, 0, 0], (len(pairs), 1))
    for s, (a, b, second) in enumerate(pairs):
        p[s * n, 1], q[s * n, 1] = a, b
        p[s * n, 2], q[s * n, 2] = 0.0, 0.5            # (never stands, whatever u)
        tokens[s] = [0, 2, 1] if second else [0, 1, 3]
    u, final = rng.random(len(pairs) * n).astype(np.float32), rng.random(len(pairs)).astype(np.float32)
    p, q = (torch.from_numpy(x).to(dtype) for x in (p, q))
    got = call([n] * len(pairs), parents.reshape(-1), tokens.reshape(-1), p, q, u, final, 3)
    clean = lambda x: np.clip(np.where(np.isnan(S.f64(x)), 0.0, S.f64(x)), 0.0, 1.0)
    stood = 0
    for s in range(len(pairs)):
        rows = slice(s * n, s * n + n)
        path, after = V.walk(n, parents[s], tokens[s], clean(p)[rows], clean(q)[rows], u[rows].astype(float),
                             float(final[s]), 3)
        assert list(got[0][s][:got[1][s]]) == path and got[2][s] == after, pairs[s]
        stood += len(path) > 1
    assert 20 < stood < len(pairs) - 20


def test_without_a_draft_model_too():
    """p at certain drafts: NaN and negative ones never stand, ones above 1 always."""
    p = np.tile([0.25, 0.25, 0.25, 0.25], (2 * len(STRANGE), 1))
    p[::2, 1] = STRANGE
    got = call([2] * len(STRANGE), [-1, 0] * len(STRANGE), [0, 1] * len(STRANGE), p, None, [0.0, 0.2] * len(STRANGE),
               [0.5] * len(STRANGE), 2)
    assert got[1].tolist() == [1, 1, 2, 1, 2, 1, 2, 2]


def test_at_the_border_behind_refusals():
    """u q Z against r, at the fp32 number nearest to r / (q Z) and its neighbours, as exact fractions have it: products
    of three are off by 2^-45, so a border must not move by 2^-25, an fp32 rounding of the product.  A second draft, behind
    one that p gives nothing, and a third behind two."""
    rng = np.random.default_rng(3)
    cases = []
    while len(cases) < 600:
        third = len(cases) % 2
        # multiples of 2^-30 that fp32 holds: every sum, and A q of A = 1, is exact in units of 2^-44
        p, q = (rng.integers(1, 1 << 24, size=6) / 2.0 ** 27 for _ in range(2))
        q[5], p[5] = 0.5, 0.0
        z = sum(max(Fraction(a) - Fraction(b), Fraction(0)) for a, b in zip(p, q))
        big_a, refused = Fraction(1), 1
        rest = [max(Fraction(a) - Fraction(b), Fraction(0)) for a, b in zip(p, q)]
        if third:
            big_a += z
            rest = [max(Fraction(a) - big_a * Fraction(b), Fraction(0)) for a, b in zip(p, q)]
            z, refused = sum(rest), 2
        # (roundings of r and Z to units: 2^-44 each of the elements, of numbers that shall be large against that)
        live = [i for i in range(5) if rest[i] > Fraction(1, 100)]
        if not live or z < Fraction(1, 20):
            continue
        x = live[0]
        mid = np.float32(float(rest[x] / (Fraction(q[x]) * z)))
        if not 0 < mid < 0.99:
            continue
        for u in (np.nextafter(mid, np.float32(0)), mid, np.nextafter(mid, np.float32(1))):
            diff = Fraction(float(u)) * Fraction(q[x]) * z / rest[x] - 1
            if abs(diff) < Fraction(1, 1 << 34):       # (6 roundings of 2^-45 against r > 1/100, and 2^-45: 2^-35)
                continue
            cases.append((p, q, x, refused, u, diff < 0))
    n = 4
    target, draft = (np.repeat(np.stack([c[i] for c in cases]), n, 0) for i in (0, 1))
    tokens, parents, u = np.full((len(cases), n), 5), np.full((len(cases), n), -1), np.full((len(cases), n), 0.9)
    for s, (_, _, x, refused, at, _) in enumerate(cases):
        parents[s, 1:2 + refused] = 0
        tokens[s, 1 + refused], u[s, 1 + refused] = x, at
        parents[s, 2 + refused:] = 1                    # (below a refused one: never tried)
    got = call([n] * len(cases), parents.reshape(-1), tokens.reshape(-1), target, draft, u.reshape(-1),
               [0.5] * len(cases), 2)
    stands = np.array([c[5] for c in cases])
    assert 0.2 < stands.mean() < 0.8
    assert np.array_equal(got[1] == 2, stands), np.flatnonzero((got[1] == 2) != stands)[:10]


# p and q of one token whose remainder p - A q, A = 4 a, is above 0 and less than a unit, and whose p and A q round to
# units so that the difference of those is -1; the other four, a and 1/4 each, leave nothing
TINY = [("0x1.7b66fap-2", "0x1.960264p-23", "0x1.11f3f8p-23"), ("0x1.70ed70p-2", "0x1.f73244p-23", "0x1.5d2b6ap-23"),
        ("0x1.72b108p-2", "0x1.ee09dap-23", "0x1.552efcp-23"), ("0x1.7563dcp-2", "0x1.a7b3f4p-23", "0x1.227eb8p-23")]


@pytest.mark.parametrize("drafts", [2, 3, 5])
def test_remainders_of_less_than_a_unit_count_as_nothing(drafts):
    """Drafts of a token that p gives nothing: the first leaves (a - 1/4 four times, p - q), the others less than a
    unit, so that what the first left stays, and a token follows."""
    n = drafts + 1
    p, q, finals, want = [], [], [], []
    for a, p1, q1 in TINY:
        a, p1, q1 = (float.fromhex(x) for x in (a, p1, q1))
        for final, token in ((0.1, 0), (0.3, 1), (0.6, 2), (0.9, 3)):
            p += [[a] * 4 + [p1, 0.0]] * n
            q += [[0.25] * 4 + [q1, 0.5]] * n
            finals.append(final)
            want.append(token)
    s = len(finals)
    got = call([n] * s, ([-1] + [0] * drafts) * s, [5] * (n * s), np.array(p), np.array(q),
               [0.5] * (n * s), finals, 2)
    assert got[1].tolist() == [1] * s and got[2].tolist() == want
