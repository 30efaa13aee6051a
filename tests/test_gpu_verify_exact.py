"""verify_drafts where its numbers are delicate: drafts tried on probabilities
that are none."""
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
