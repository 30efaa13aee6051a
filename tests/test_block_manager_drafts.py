"""The block manager through a step of drafted tokens: slots for all of them, the
refused ones' blocks back."""
import numpy as np
import pytest

from paged_kv_cache_177_gb300.block_manager import BlockManager, NoFreeBlocks


def test_drafts_take_slots_and_give_them_back():
    m = BlockManager(8)
    m.allocate(0, 14)
    slots, cow = m.append_slots(0, 21)                     # 35 tokens: two blocks more
    table = m.block_table(0)
    assert slots == [table[p // 16] * 16 + p % 16 for p in range(14, 35)] and cow is None
    assert len(table) == 3 and m.num_free == 5
    m.truncate(0, 16)                                      # two drafts kept: the first block is full, no other is needed
    assert m.block_table(0) == table[:1] and m.context_len(0) == 16 and m.num_free == 7
    m.check_invariants()
    slot, cow = m.append_slot(0)
    assert slot % 16 == 0 and cow is None and len(m.block_table(0)) == 2
    m.truncate(0, 17)                                      # nothing refused
    m.check_invariants()
    m.truncate(0, 0)
    assert m.block_table(0) == [] and m.num_free == 8
    m.check_invariants()
    assert m.append_slots(0, 0) == ([], None)


def test_a_shared_block_is_copied_once():
    m = BlockManager(8)
    m.allocate(0, 20)
    m.fork(0, 1)
    shared = m.block_table(0)
    slots, cow = m.append_slots(1, 14)                     # 34 tokens: a copy of the second block, and a third
    table = m.block_table(1)
    assert cow == (shared[1], table[1]) and table[0] == shared[0] and table[1] != shared[1] and len(table) == 3
    assert slots[0] == table[1] * 16 + 4
    m.check_invariants()
    m.truncate(1, 10)                                      # back into the block that is still shared
    assert m.block_table(1) == shared[:1]
    m.check_invariants()
    slots, cow = m.append_slots(1, 1)                      # which a new token must not be written to
    assert cow == (shared[0], m.block_table(1)[0]) and slots == [m.block_table(1)[0] * 16 + 10]
    m.check_invariants()


def test_all_or_nothing():
    m = BlockManager(3)
    m.allocate(0, 20)
    m.fork(0, 1)
    before = m.block_table(1)
    with pytest.raises(NoFreeBlocks):                      # the copy and two more, one is free
        m.append_slots(1, 30)
    assert m.block_table(1) == before and m.context_len(1) == 20 and m.num_free == 1
    m.check_invariants()
    m.append_slots(1, 12)                                  # the copy alone
    m.check_invariants()
    for n in (-1, 33):
        with pytest.raises(ValueError):
            m.truncate(1, n)
    with pytest.raises(ValueError):
        m.append_slots(1, -1)


def test_random_steps_keep_the_pool_whole():
    rng = np.random.default_rng(2)
    m = BlockManager(60)
    for s in range(4):
        m.allocate(s, int(rng.integers(0, 40)))
    for step in range(300):
        s = int(rng.integers(4))
        try:
            slots, _ = m.append_slots(s, int(rng.integers(0, 33)))
        except NoFreeBlocks:
            m.truncate(s, int(rng.integers(0, m.context_len(s) + 1)))
            m.check_invariants()
            continue
        n = len(slots)
        base, table = m.context_len(s) - n, m.block_table(s)
        assert slots == [table[p // 16] * 16 + p % 16 for p in range(base, base + n)]
        m.check_invariants()
        m.truncate(s, base + int(rng.integers(0, n + 1)))
        m.check_invariants()
