"""Steps of speculative decoding on the host's block manager."""
import numpy as np
import pytest
import torch

from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


def test_steps_of_drafts_on_the_block_manager():
    """Slots, tables and lengths from the host's block manager: drafts appended, a path accepted in two layers, the rest
    given back, over several steps; after each the caches hold the accepted rows in order."""
    from paged_kv_cache_177_gb300.block_manager import BlockManager
    b = S.lib()
    rng = np.random.default_rng(9)
    torch.manual_seed(9)
    hkv, d, layers, seqs = 2, 64, 2, 3
    m = BlockManager(24, order=rng.permutation(24))
    caches = [torch.zeros(24, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2 * layers)]
    rows = {}                                    # (sequence) -> accepted rows, [cache][token]
    for s in range(seqs):
        m.allocate(s)
        rows[s] = [[] for _ in caches]
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    for step in range(6):
        ns = [int(rng.integers(1, 24)) for _ in range(seqs)]
        slots = [x for s in range(seqs) for x in m.append_slots(s, ns[s])[0]]
        new = [torch.randn(sum(ns), hkv, d, device="cuda").bfloat16() for _ in caches]
        for layer in range(layers):
            b.kv_append(new[layer], new[layers + layer], torch.tensor(slots, device="cuda"), caches[layer],
                        caches[layers + layer])
        tables, lens = m.tables_array(list(range(seqs)))
        paths = [np.sort(rng.choice(n, size=int(rng.integers(0, min(n, 5) + 1)), replace=False)) for n in ns]
        accepted = np.zeros((seqs, 5), dtype=np.int32)
        for s, p in enumerate(paths):
            accepted[s, :len(p)] = p
        start = np.concatenate([[0], np.cumsum(ns)])
        out = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        b.kv_accept_layers(caches[:layers], caches[layers:], i32(tables), i32(lens), i32(start), i32(accepted),
                           i32([len(p) for p in paths]), out)
        for s, length in enumerate(out.tolist()):
            for c in range(len(caches)):
                rows[s][c] += [new[c][start[s] + j] for j in paths[s]]
            m.truncate(s, length)
            m.check_invariants()
            table = m.block_table(s)
            assert len(rows[s][0]) == length
            for c, cache in enumerate(caches):
                for p, row in enumerate(rows[s][c]):
                    assert torch.equal(cache[table[p // 16], :, p % 16], row), (step, s, p)
    assert b.device_error() == 0
