"""The copy pairs of one step obey pa_block_copy's rule (distinct targets, none of them a source)
and give every sequence its own data, whatever was forked, made private, cut, freed or appended to
before they are taken."""
import random

import pytest

from paged_kv_cache_335_b200.block_manager import BlockManager, PoolExhausted


def _take(m):
    pairs = m.take_copies().tolist()
    dst = [d for _, d in pairs]
    assert len(set(dst)) == len(dst), f"a block is the target of two copies: {pairs}"
    assert not set(dst) & {s for s, _ in pairs}, f"a target is a source too: {pairs}"
    return pairs


def test_a_copy_of_a_copy_comes_from_the_first_source():
    m = BlockManager(10, 16)
    a = m.new_sequence(32)
    b = m.fork(a)
    m.unshare(b)
    c = m.fork(b)                               # before b's copies were made
    m.unshare(c)
    assert sorted(_take(m)) == sorted([list(p) for p in zip(a.table, b.table)] + [list(p) for p in zip(a.table, c.table)])


def test_a_freed_target_is_no_target_any_more():
    m = BlockManager(8, 16)
    a = m.new_sequence(32)
    b = m.fork(a)
    m.unshare(b)
    gone = list(b.table)
    m.free(b)
    c = m.fork(a)
    m.unshare(c)
    assert set(c.table) & set(gone)
    assert sorted(_take(m)) == sorted(list(p) for p in zip(a.table, c.table))


def test_a_freed_source_is_no_target_before_its_copy():
    m = BlockManager(6, 16)
    a, x = m.new_sequence(16), m.new_sequence(16)
    b, y = m.fork(a), m.fork(x)
    m.unshare(b)                                # a's block -> b's
    source = a.table[0]
    m.free(a)
    m.unshare(y)
    assert y.table != [source]
    pairs = _take(m)
    assert [source, b.table[0]] in pairs and [x.table[0], y.table[0]] in pairs
    z = m.fork(x)
    m.unshare(z)                                # after its copy it is a block like any other
    assert z.table == [source]


def test_no_target_left_changes_nothing():
    m = BlockManager(4, 16)
    a, x = m.new_sequence(16), m.new_sequence(16)
    b, y = m.fork(a), m.fork(x)
    m.unshare(b)
    spare = m.new_sequence(16)                  # the pool's last block
    m.free(a)                                   # its block still has to be copied
    with pytest.raises(PoolExhausted):
        m.unshare(y)
    assert y.table == x.table and m.num_free == 1 and list(m.refcount[x.table]) == [2]
    _take(m)
    assert m.unshare(y) == 1 and spare.length == 16


@pytest.mark.parametrize("seed", range(40))
def test_any_order_of_calls(seed):
    rng = random.Random(seed)
    bs = 4
    m = BlockManager(24, bs, order=random.Random(seed).sample(range(24), 24))
    pool = {b: [None] * bs for b in range(24)}
    seqs = []                                   # [sequence, its tokens, {position: token} not yet written]
    count = 0

    def flush():
        fresh = {d: list(pool[s]) for s, d in _take(m)}
        pool.update(fresh)
        for s, _, writes in seqs:
            for p, v in writes.items():
                pool[s.table[p // bs]][p % bs] = v
            writes.clear()
        for s, tokens, _ in seqs:
            assert [pool[s.table[p // bs]][p % bs] for p in range(s.length)] == tokens

    for _ in range(300):
        op = rng.choice(["new", "fork", "unshare", "unshare", "append", "append", "truncate", "free", "flush"])
        pick = rng.choice(seqs) if seqs else None
        try:
            if op == "new" and len(seqs) < 6:
                seqs.append([m.new_sequence(0), [], {}])
            elif op == "fork" and pick and not pick[2] and len(seqs) < 6:
                seqs.append([m.fork(pick[0]), list(pick[1]), {}])
            elif op == "unshare" and pick:
                m.unshare(pick[0])
            elif op == "append" and pick:
                m.append_slot(pick[0])
                count += 1
                pick[2][pick[0].length - 1] = count
                pick[1].append(count)
            elif op == "truncate" and pick:
                n = rng.randint(0, pick[0].length)
                m.truncate(pick[0], n)
                del pick[1][n:]
                for p in [p for p in pick[2] if p >= n]:
                    del pick[2][p]
            elif op == "free" and pick:
                m.free(pick[0])
                seqs.remove(pick)
            elif op == "flush":
                flush()
        except PoolExhausted:
            flush()
            if seqs and not m.num_free:
                m.free(seqs[0][0])
                seqs.pop(0)
    flush()
    for s, _, _ in seqs:
        m.free(s)
    assert m.num_free == 24 and not m.refcount.any()
