"""Host side of an eviction: private blocks before it, freed blocks after it."""
import pytest

from paged_kv_cache_335_b200.block_manager import BlockManager, PoolExhausted


def test_truncate_frees_the_blocks_behind():
    m = BlockManager(10, 16)
    s = m.new_sequence(70)                      # 5 blocks
    table = list(s.table)
    m.truncate(s, 33)
    assert s.table == table[:3] and s.length == 33 and m.num_free == 7
    assert m.append_slot(s) == table[2] * 16 + 1
    m.truncate(s, 32)
    assert len(s.table) == 2
    m.truncate(s, 0)
    assert s.table == [] and m.num_free == 10
    for bad in (-1, 1):
        with pytest.raises(ValueError):
            m.truncate(s, bad)


def test_truncate_keeps_shared_blocks_alive():
    m = BlockManager(10, 16)
    a = m.new_sequence(48)
    b = m.fork(a)
    m.truncate(a, 16)
    assert m.num_free == 7 and b.length == 48
    m.free(b)
    assert m.num_free == 9
    m.free(a)
    assert m.num_free == 10


def test_unshare_copies_every_shared_block():
    m = BlockManager(8, 16)
    a = m.new_sequence(40)                      # 3 blocks
    assert m.unshare(a) == 0
    b = m.fork(a)
    assert m.unshare(b) == 3
    assert not set(a.table) & set(b.table) and list(m.refcount[a.table]) == [1, 1, 1]
    assert m.take_copies().tolist() == [list(p) for p in zip(a.table, b.table)]
    c = m.fork(b)
    with pytest.raises(PoolExhausted):          # 3 to copy, 2 free: nothing is changed
        m.unshare(c)
    assert c.table == b.table and m.num_free == 2 and m.take_copies().size == 0
