"""Steps of a serving loop with the calls around transformed scores: a prompt
prefilled through a layer with capped scores and a window, forked into
requests that share its blocks, chains of drafts attended, verified and
accepted on the host's block manager, the batch decoded over the common
prefix and through the layer; every attention against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests import score_helpers as H
from tests import serving_helpers as S
from tests import verify_helpers as V

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def test_a_prompt_its_forks_and_their_drafts():
    from paged_kv_cache_177_gb300.block_manager import BlockManager
    B = S.lib()
    B.device_error()
    rng = np.random.default_rng(21)
    torch.manual_seed(21)
    hq, hkv, d, vocab, prompt, seqs, most = 8, 2, 64, 97, 333, 5, 6
    layer = dict(softcap=6.0, window=200)
    scale = 0.3
    m = BlockManager(80, order=rng.permutation(80))
    k_cache, v_cache = (torch.full((80, hkv, 16, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    head = torch.randn(hq * d, vocab, device="cuda") * 0.2
    rows = lambda n, heads: torch.randn(n, heads, d, device="cuda").to(BF)

    def seen(s, n):
        """A sequence's n rows in order, from the cache."""
        table = np.asarray(m.block_table(s))
        return [S.gather(np.nan_to_num(S.f64(c)), table, n, 80) for c in (k_cache, v_cache)]

    # the prompt, its first 64 tokens seen from both sides
    m.allocate(0, prompt)
    slots = [b * 16 + o for b in m.block_table(0) for o in range(16)][:prompt]
    B.kv_append(rows(prompt, hkv), rows(prompt, hkv), torch.tensor(slots, device="cuda"), k_cache, v_cache)
    tables, lens = m.tables_array([0])
    q = rows(prompt, hq)
    out = torch.empty_like(q)
    B.paged_prefill_attention_scored(out, q, k_cache, v_cache, i32(tables), i32(lens), i32([0, prompt]), scale,
                                     prefix_lens=i32([64]), **layer)
    want, bound = H.attend(S.f64(q), *seen(0, prompt), scale, np.arange(prompt), 6.0, None, 200, 64)
    S.close(out, want, bound, "prompt")
    for s in range(1, seqs):
        m.fork(0, s)

    kept = [prompt] * seqs
    grew = 0
    for step in range(5):
        # a chain of drafts behind each request, row 0 its last chosen token
        ns = [int(rng.integers(1, 9)) for _ in range(seqs)]
        slots, copies = [], []
        for s in range(seqs):
            got, cow = m.append_slots(s, ns[s])
            slots += got
            copies += [cow] if cow else []
        if copies:
            B.copy_blocks(k_cache, v_cache, torch.tensor(copies, dtype=torch.int64, device="cuda"))
        total = sum(ns)
        B.kv_append(rows(total, hkv), rows(total, hkv), torch.tensor(slots, device="cuda"), k_cache, v_cache)
        tables, lens = m.tables_array(list(range(seqs)))
        start = np.concatenate([[0], np.cumsum(ns)])
        q = rows(total, hq)
        out = torch.empty_like(q)
        B.paged_prefill_attention_scored(out, q, k_cache, v_cache, i32(tables), i32(lens), i32(start), scale, **layer)
        for s in range(seqs):
            r = slice(start[s], start[s + 1])
            want, bound = H.attend(S.f64(q[r]), *seen(s, lens[s]), scale, np.arange(lens[s] - ns[s], lens[s]), 6.0, None, 200)
            S.close(out[r], want, bound, f"step {step}, drafts of {s}")
        # what the layer's outputs say, and a draft model near it
        logits = out.float().view(total, -1) @ head
        target = torch.softmax(logits, -1)
        near = torch.softmax(logits + 0.3 * torch.randn_like(logits), -1)
        parents = np.concatenate([np.arange(n) - 1 for n in ns])
        tokens = np.zeros(total, dtype=np.int64)
        for s in range(seqs):
            for i in range(1, ns[s]):
                tokens[start[s] + i] = int(torch.multinomial(near[start[s] + i - 1], 1))
        u, final = torch.rand(total, device="cuda"), torch.rand(seqs, device="cuda")
        accepted = torch.zeros(seqs, most, dtype=torch.int32, device="cuda")
        count, chosen = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(seqs, dtype=torch.int64, device="cuda")
        args = (torch.from_numpy(tokens).cuda(), i32(parents), i32(start))
        B.verify_drafts(accepted, count, chosen, *args, target, u, final, draft_probs=near)
        ref = V.walk_all(args[2], args[1], args[0], target, near, u, final, most)
        assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip((accepted, count, chosen), ref))
        # the accepted ones stay, the others' blocks go back
        new_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        B.kv_accept_layers([k_cache], [v_cache], i32(tables), i32(lens), i32(start), accepted, count, new_lens)
        for s, n in enumerate(new_lens.tolist()):
            assert n == kept[s] + int(count[s])
            grew += n - kept[s] > 1
            kept[s] = n
            m.truncate(s, n)
        m.check_invariants()
        # a decode step through the layer, and one over the shared prompt
        tables, lens = m.tables_array(list(range(seqs)))
        q = rows(seqs, hq)
        one, all_ = torch.empty_like(q), torch.empty_like(q)
        B.paged_decode_attention_scored(one, q, k_cache, v_cache, i32(tables), i32(lens), scale, **layer)
        B.paged_decode_attention_common_prefix(all_, q, k_cache, v_cache, i32(tables), i32(lens), scale, i32([0, seqs]),
                                               i32([prompt // 16]))
        for s in range(seqs):
            assert tables[s, :prompt // 16].tolist() == tables[0, :prompt // 16].tolist()
            kv = seen(s, lens[s])
            want, bound = H.attend(S.f64(q[s:s + 1]), *kv, scale, [lens[s] - 1], 6.0, None, 200)
            S.close(one[s:s + 1], want, bound, f"step {step}, decode of {s}")
            want, bound = H.attend(S.f64(q[s:s + 1]), *kv, scale, [lens[s] - 1])
            S.close(all_[s:s + 1], want, bound, f"step {step}, common prefix of {s}")
    assert grew > 0 and B.device_error() == 0


def test_a_step_in_one_graph():
    """Tree attention, verification and acceptance captured together, replayed with other random numbers."""
    B = S.lib()
    B.device_error()
    torch.manual_seed(22)
    rng = np.random.default_rng(22)
    hq, hkv, d, vocab, seqs = 4, 2, 64, 50, 3
    ns, ctx = [7, 5, 9], [40, 90, 16]
    lens = [a + b for a, b in zip(ns, ctx)]
    tables, nb = S.layout(rng, lens)
    start = np.concatenate([[0], np.cumsum(ns)])
    k0, v0 = (torch.randn(nb, hkv, 16, d, device="cuda").to(BF) for _ in range(2))
    k, v = k0.clone(), v0.clone()
    parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)] for n in ns])
    q = torch.randn(sum(ns), hq, d, device="cuda").to(BF)
    head = torch.randn(hq * d, vocab, device="cuda") * 0.2
    tokens = torch.from_numpy(rng.integers(0, vocab, sum(ns))).cuda()
    tt, lt, st, pt = i32(tables), i32(lens), i32(start), i32(parents)
    u, final = torch.rand(sum(ns), device="cuda"), torch.rand(seqs, device="cuda")
    mask = torch.zeros(sum(ns), 1, dtype=torch.int64, device="cuda")
    out, target = torch.empty_like(q), torch.empty(sum(ns), vocab, device="cuda")
    res = (torch.zeros(seqs, 8, dtype=torch.int32, device="cuda"), torch.zeros(seqs, dtype=torch.int32, device="cuda"),
           torch.zeros(seqs, dtype=torch.int64, device="cuda"))
    new_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    ptrs = (B.layer_pointers([k]), B.layer_pointers([v]))
    ws = torch.zeros(max(16, B.tree_workspace_bytes(seqs, hq, hkv, d, 9, max(lens))), dtype=torch.uint8, device="cuda")

    def step():
        B.tree_masks(pt, st, 9, out=mask)
        B.paged_tree_attention(out, q, k, v, tt, lt, st, mask, 0.3, max_query_len=9, max_context_len=max(lens), workspace=ws)
        target.copy_(torch.softmax(out.float().view(sum(ns), -1) @ head, -1))
        B.verify_drafts(*res, tokens, pt, st, target, u, final, max_query_len=9)
        B.kv_accept_layers([k], [v], tt, lt, st, res[0], res[1], new_lens, ptrs=ptrs)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    most = 0
    for _ in range(4):
        k.copy_(k0)
        v.copy_(v0)
        u.uniform_(0, 0.02)      # (certain drafts of 50 tokens: about half stand)
        final.uniform_()
        graph.replay()
        ref = V.walk_all(st, pt, tokens, target, None, u, final, 8)
        assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(res, ref))
        for s in range(seqs):
            path = ref[0][s][:ref[1][s]]
            most = max(most, len(path))
            assert int(new_lens[s]) == ctx[s] + len(path)
            for j, r in enumerate(path):
                at, to = ctx[s] + int(r), ctx[s] + j
                assert torch.equal(k[tables[s, to // 16], :, to % 16], k0[tables[s, at // 16], :, at % 16])
    assert most > 1 and B.device_error() == 0
