"""paged_decode_attention_common_prefix against attention in 64 bits: groups
of any size over prefixes of any length, their own blocks behind, poisoned
caches."""
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


def make(seed, groups, lens, shared, hq, hkv, d, gain=1.0):
    """groups: first sequence of each and the end; shared: blocks that each group's tables have in common.  Everything
    that is no token of a sequence is NaN or infinite, unused table entries are out of range."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 16) for n in lens]
    nb = sum(need) + 3
    perm = list(rng.permutation(nb))
    tables = np.full((len(lens), max(1, max(need))), 1 << 30, dtype=np.int32)
    dead = np.ones((nb, 16), dtype=bool)
    for s, n in enumerate(lens):
        z = next((z for z in range(len(groups) - 1) if groups[z] <= s < groups[z + 1]), None)
        lead = groups[z] if z is not None else s
        both = min(shared[z], need[s], need[lead]) if z is not None and lead != s else 0
        tables[s, :both] = tables[lead, :both]
        for j in range(both, need[s]):
            tables[s, j] = perm.pop()
        for t in range(n):
            dead[tables[s, t // 16], t % 16] = False
    k = torch.from_numpy(rng.standard_normal((nb, hkv, 16, d)).astype(np.float32) * gain).to(BF)
    v = torch.from_numpy(rng.standard_normal((nb, hkv, 16, d)).astype(np.float32)).to(BF)
    kn, vn = S.f64(k), S.f64(v)
    rows = [(S.gather(kn, tables[s], n, nb), S.gather(vn, tables[s], n, nb)) for s, n in enumerate(lens)]
    where = torch.from_numpy(dead)[:, None, :, None].expand_as(k)
    k = torch.where(where, torch.tensor(float("nan"), dtype=BF), k)
    v = torch.where(where, torch.tensor(float("inf"), dtype=BF), v)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, d)).astype(np.float32)).to(BF)
    return q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(tables).cuda(), rows


def compare(out, q, rows, lens, scale, what=""):
    got, qf = S.f64(out), S.f64(q)
    for s, n in enumerate(lens):
        want, bound = H.attend(qf[s:s + 1], *rows[s], scale, [n - 1])
        S.close(got[s:s + 1], want, bound, f"{what} sequence {s} of {n}")


def run(seed, groups, lens, shared, hq, hkv, d, gain=1.0, **kw):
    B = S.lib()
    B.device_error()
    q, k, v, tables, rows = make(seed, groups, lens, shared, hq, hkv, d, gain)
    out = torch.full_like(q, float("nan"))
    scale = d ** -0.5
    B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), scale, i32(groups), i32(shared), **kw)
    compare(out, q, rows, lens, scale)
    assert B.device_error() == 0
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 4), (9, 3), (12, 3), (16, 2), (32, 2), (7, 1)])
def test_every_group_width(d, hq, hkv):
    lens = [100, 97, 200, 96, 111, 300, 130, 129]
    run(d + hq, [0, 8], lens, [6], hq, hkv, d)
    run(d + hq + 1, [0, 3, 8], lens, [4, 6], hq, hkv, d)


@pytest.mark.parametrize("shared", [0, 1, 3, 4, 7, 8, 9, 40, 130])
def test_prefixes_of_every_length(shared):
    """Up to where rows see few keys, chunks' ends, and enough chunks to be cut among workers."""
    rng = np.random.default_rng(shared)
    lens = [16 * shared + int(x) for x in rng.integers(1, 70, 20)]
    run(shared, [0, 20], lens, [shared], 8, 2, 64)
    run(shared + 1, [0, 1, 6, 20], lens, [shared, shared, shared], 4, 4, 128)


@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 64, 65, 130, 200])
def test_groups_of_every_size(seqs):
    """One tile of rows, two, and several sets of two."""
    rng = np.random.default_rng(seqs)
    lens = [160 + int(x) for x in rng.integers(0, 40, seqs)]
    run(seqs, [0, seqs], lens, [10], 8, 2, 64)
    run(seqs, [0, seqs], lens, [10], 4, 4, 64)


@pytest.mark.parametrize("seqs,hq,hkv", [(3, 15, 5), (23, 15, 5), (1, 7, 1), (5, 3, 1), (7, 5, 5)])
def test_an_odd_number_of_rows(seqs, hq, hkv):
    """The workspace's parts stay aligned whatever lies before them; whole prefixes, and prefixes cut among workers."""
    rng = np.random.default_rng(seqs)
    for d in (64, 128):
        for shared in (2, 3, 70):
            lens = [16 * shared + int(x) for x in rng.integers(0, 13, seqs)]
            run(seqs, [0, seqs], lens, [shared], hq, hkv, d)
            if seqs > 1:                       # (no more groups than sequences)
                run(seqs, [0, (seqs + 1) // 2, seqs], lens, [shared, shared], hq, hkv, d)


def test_contexts_that_end_with_the_prefix():
    """Nothing behind the prefix: the output is the prefix' alone, cut or not."""
    run(1, [0, 5], [160] * 5, [10], 8, 2, 64)
    run(2, [0, 5], [160, 160, 161, 175, 160], [10], 4, 4, 128)
    run(3, [0, 4], [2048, 2048, 2050, 2048], [128], 8, 2, 64)
    run(4, [0, 4], [160, 170, 180, 1000], [30], 8, 2, 64)       # more than the shortest member has


def test_empty_contexts_and_sequences_in_no_group():
    run(5, [0, 3], [0, 50, 60], [3], 8, 2, 64)                   # an empty member: nothing is shared
    run(6, [2, 5, 5, 9], [40, 0, 130, 140, 135, 70, 66, 69, 80, 33, 0, 16], [8, 2, 4], 8, 2, 64)
    run(7, [0, 0], [40, 50], [2], 4, 2, 64)
    q, k, v, tables, rows = make(8, [0], [40, 50], [], 4, 2, 64)
    out = torch.empty_like(q)
    S.lib().paged_decode_attention_common_prefix(out, q, k, v, tables, i32([40, 50]), 0.1, i32([0]), i32([]))
    compare(out, q, rows, [40, 50], 0.1)


def test_long_prefixes_and_large_scores():
    rng = np.random.default_rng(9)
    lens = [4096 + int(x) for x in rng.integers(1, 600, 40)]
    run(9, [0, 40], lens, [256], 8, 2, 128)
    run(10, [0, 10, 40], lens, [255, 100], 16, 1, 64, gain=6.0)


def test_many_groups():
    rng = np.random.default_rng(11)
    lens = list(rng.integers(48, 300, 120))
    run(11, list(range(0, 121, 3)), lens, [3] * 40, 8, 2, 64)


def test_one_workspace_in_turn_with_other_calls():
    B = S.lib()
    ws = torch.zeros(B.common_prefix_workspace_bytes(30, 8, 2, 64), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(12)
    lens = [480 + int(x) for x in rng.integers(1, 300, 30)]
    for _ in range(2):
        run(12, [0, 30], lens, [30], 8, 2, 64, workspace=ws)
        q, k, v, tables, rows = make(13, [0], lens, [], 8, 2, 64)
        a = B.paged_decode_attention(torch.empty_like(q), q, k, v, tables, i32(lens), 0.125, workspace=ws)
        compare(a, q, rows, lens, 0.125)
        assert int(ws[:B.DECODE_COUNTER_BYTES].max()) == 0
    a = run(12, [0, 30], lens, [30], 8, 2, 64, workspace=ws)
    assert torch.equal(a, run(12, [0, 30], lens, [30], 8, 2, 64))           # bit-repeatable


def test_what_is_not_finite_in_the_prefix_reaches_all_of_the_group():
    """In every row of the group its element is what a sum over it is; other groups keep theirs."""
    B = S.lib()
    for shared in (3, 20):
        lens = [16 * shared + 20] * 6
        q, k, v, tables, rows = make(14, [0, 3, 6], lens, [shared, shared], 4, 2, 64)
        v[tables[0, 1], 1, 5, 9] = float("inf")
        v[tables[0, 2], 1, 5, 11] = float("nan")
        out = torch.empty_like(q)
        B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.125, i32([0, 3, 6]), i32([shared] * 2))
        got = S.f64(out)
        assert np.all(got[:3, 2:, 9] == np.inf) and np.all(np.isnan(got[:3, 2:, 11]))
        got[:3, 2:, [9, 11]] = 0
        for s in range(6):
            want, bound = H.attend(S.f64(q[s:s + 1]), *rows[s], 0.125, [lens[s] - 1])
            if s < 3:
                want[:, 2:, [9, 11]] = 0
            S.close(got[s:s + 1], want, bound)


def test_bad_pages_and_groups():
    B = S.lib()
    lens = [100, 110, 120, 90]
    q, k, v, tables, rows = make(15, [0, 4], lens, [5], 8, 2, 64)
    B.device_error()
    tables[0:4, 2] = -1
    tables[3, 5] = 1 << 20
    out = torch.empty_like(q)
    B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.125, i32([0, 4]), i32([5]))
    for s in range(4):
        for a in rows[s]:
            a[32:48] = 0.0
            if s == 3:
                a[80:96] = 0.0
    compare(out, q, rows, lens, 0.125)
    assert B.device_error() == B.DEVERR_BLOCK_ID
    # a group past the bound, one past the batch, one of fewer than none: flagged, nothing shared
    q, k, v, tables, rows = make(16, [0, 4], lens, [5], 8, 2, 64)
    for starts, most in (([0, 4], 3), ([0, 5], 9), ([3, 1], 4), ([-1, 4], 9)):
        out.fill_(float("nan"))
        B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.125, i32(starts), i32([5]),
                                               max_group_size=most)
        compare(out, q, rows, lens, 0.125)
        assert B.device_error() == B.DEVERR_LENGTH
    B.paged_decode_attention_common_prefix(out, q, k, v, tables, i32(lens), 0.125, i32([0, 4]), i32([-2]))
    compare(out, q, rows, lens, 0.125)


def test_captured_and_on_another_stream():
    B = S.lib()
    lens = [700, 650, 655, 641, 1000]
    q, k, v, tables, rows = make(17, [0, 5], lens, [40], 8, 2, 64)
    out, lt, gs, sb = torch.empty_like(q), i32(lens), i32([0, 5]), i32([40])
    ws = torch.zeros(B.common_prefix_workspace_bytes(5, 8, 2, 64), dtype=torch.uint8, device="cuda")
    call = lambda **kw: B.paged_decode_attention_common_prefix(out, q, k, v, tables, lt, 0.125, gs, sb, max_group_size=5,
                                                               max_context_len=1000, **kw)
    call(workspace=ws)
    compare(out, q, rows, lens, 0.125)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(workspace=ws)
    for _ in range(3):
        q.copy_(torch.randn_like(q))
        graph.replay()
        compare(out, q, rows, lens, 0.125)
    side = torch.cuda.Stream()
    q.copy_(torch.randn_like(q))
    out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    compare(out, q, rows, lens, 0.125)
