"""Far ends: caches and rows of probabilities past 2^31 elements, batches past
a launch's usual size."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests import verify_helpers as V

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


@pytest.fixture(scope="module")
def far_pool():
    """Two caches of 2.2e9 elements whose last blocks are filled."""
    torch.manual_seed(3)
    nb, hkv, d, used = 135000, 8, 128, 64
    k, v = (torch.empty(nb, hkv, 16, d, dtype=BF, device="cuda") for _ in range(2))
    k[-used:] = torch.randn(used, hkv, 16, d, device="cuda").to(BF)
    v[-used:] = torch.randn(used, hkv, 16, d, device="cuda").to(BF)
    assert k.numel() > 1 << 31
    yield k, v, nb - used
    del k, v
    torch.cuda.empty_cache()


def rows_of(k, v, table, n):
    t = np.arange(n)
    at = torch.from_numpy(table[t // 16].astype(np.int64)).cuda()
    return [S.f64(c[at, :, torch.from_numpy(t % 16).cuda()]) for c in (k, v)]


def test_caches_past_two_to_the_thirty_first(far_pool):
    B = S.lib()
    B.device_error()
    k, v, first = far_pool
    lens = [300, 290]
    tables = np.stack([first + np.arange(19), first + np.concatenate([np.arange(8), 30 + np.arange(11)])]).astype(np.int32)
    kv = [rows_of(k, v, tables[s], lens[s]) for s in range(2)]
    q = torch.randn(2, 16, 128, device="cuda").to(BF)
    out = torch.empty_like(q)
    B.paged_decode_attention_scored(out, q, k, v, i32(tables), i32(lens), 0.1, softcap=9.0, window=100)
    for s in range(2):
        want, bound = H.attend(S.f64(q[s:s + 1]), *kv[s], 0.1, [lens[s] - 1], 9.0, None, 100)
        S.close(out[s:s + 1], want, bound)
    B.paged_decode_attention_common_prefix(out, q, k, v, i32(tables), i32(lens), 0.1, i32([0, 2]), i32([8]))
    for s in range(2):
        want, bound = H.attend(S.f64(q[s:s + 1]), *kv[s], 0.1, [lens[s] - 1])
        S.close(out[s:s + 1], want, bound)
    q = torch.randn(200, 16, 128, device="cuda").to(BF)
    out = torch.empty_like(q)
    keep = v[tables[0, 18], 3, 5, 7].clone()
    v[tables[0, 18], 3, 5, 7] = float("inf")           # position 293, seen by the last rows only
    B.paged_prefill_attention_scored(out, q, k, v, i32(tables[:1]), i32(lens[:1]), i32([0, 200]), 0.1, softcap=9.0)
    v[tables[0, 18], 3, 5, 7] = keep
    want, bound = H.attend(S.f64(q), *kv[0], 0.1, np.arange(100, 300), 9.0)
    got = S.f64(out)
    assert np.all(got[193:, 6:8, 7] == np.inf)
    got[193:, 6:8, 7] = want[193:, 6:8, 7]
    S.close(got, want, bound)
    assert B.device_error() == 0


def test_probabilities_past_two_to_the_thirty_first():
    B = S.lib()
    rows, vocab = 33000, 65537
    target = torch.zeros(rows, vocab, dtype=BF, device="cuda")
    assert target.numel() > 1 << 31
    ns = [rows - 6, 6]                                  # (the first sequence has more rows than fit: flagged)
    start, parents, tokens, small, _, u, final = V.trees(4, [6], vocab, False, BF, back=2)
    target[-6:] = small
    pad = lambda t, fill: torch.cat([torch.full((rows - 6,), fill, dtype=t.dtype, device="cuda"), t])
    out = (torch.zeros(2, 6, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
           torch.zeros(2, dtype=torch.int64, device="cuda"))
    B.device_error()
    B.verify_drafts(*out, pad(tokens, 0), pad(parents, -1), i32([0, ns[0], rows]), target, pad(u, 0.5),
                    torch.cat([final, final]), max_query_len=6)
    want = V.walk_all(start, parents, tokens, small, None, u, final, 6)
    assert np.array_equal(out[0][1].cpu().numpy(), want[0][0]) and int(out[1][1]) == want[1][0]
    assert int(out[2][1]) == want[2][0]
    assert int(out[1][0]) == 0 and int(out[2][0]) == -1 and B.device_error() == B.DEVERR_LENGTH


def test_batches_of_thousands():
    B = S.lib()
    B.device_error()
    rng = np.random.default_rng(5)
    seqs = 9000                                         # past the persistent kernel's table of sequences
    lens = [int(x) for x in rng.integers(0, 24, seqs)]
    k, v, tables, kr, vr = H.paged(6, lens, 1, 64, BF, window=10)
    q = torch.randn(seqs, 2, 64, device="cuda").to(BF)
    out = torch.empty_like(q)
    B.paged_decode_attention_scored(out, q, k, v, tables, i32(lens), 0.125, softcap=5.0, window=10)
    some = rng.integers(0, seqs, 300)
    for s in some:
        want, bound = H.attend(S.f64(q[s:s + 1]), kr[s], vr[s], 0.125, [lens[s] - 1], 5.0, None, 10)
        S.close(out[s:s + 1], want, bound)
    ns = [min(n, 3) for n in lens]
    start = np.concatenate([[0], np.cumsum(ns)])
    k, v, tables, kr, vr = H.paged(7, lens, 1, 64, BF)
    q = torch.randn(start[-1], 2, 64, device="cuda").to(BF)
    out = torch.empty_like(q)
    B.paged_prefill_attention_scored(out, q, k, v, tables, i32(lens), i32(start), 0.125, softcap=5.0, window=10)
    for s in some:
        want, bound = H.attend(S.f64(q[start[s]:start[s + 1]]), kr[s], vr[s], 0.125, np.arange(lens[s] - ns[s], lens[s]), 5.0, None, 10)
        S.close(out[start[s]:start[s + 1]], want, bound)
    with pytest.raises(B.PagedKVError):
        big = torch.zeros(8193, 2, 64, dtype=BF, device="cuda")
        B.paged_decode_attention_common_prefix(big, big, k, v, torch.zeros(8193, 1, dtype=torch.int32, device="cuda"),
                                               torch.zeros(8193, dtype=torch.int32, device="cuda"), 0.1, i32([0, 1]), i32([0]))
    assert B.device_error() == 0
