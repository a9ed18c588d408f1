"""Copy lists of the block manager: the pairs of one list are copied at the
same time, so no destination may be a source or another pair's destination,
however full the pool is."""
import numpy as np
import pytest

from paged_kv_cache_408_b200.runtime import (BlockAllocator, KVManager, OutOfBlocksError, PrefixCache, Scheduler,
                                             SchedulerConfig, Sequence, check_invariants)


def cached_sequence(blocks, tokens):
    """A sequence whose full blocks the prefix cache names, in a pool of `blocks`."""
    alloc = BlockAllocator(blocks)
    cache, kv = PrefixCache(alloc), KVManager(alloc)
    s = Sequence(0, tokens, 4, tokens, tokens, False, [alloc.alloc() for _ in range((tokens + 15) // 16)])
    cache.insert(np.arange(tokens), s.block_table)
    return alloc, cache, kv, s


def check_pairs(pairs):
    src, dst = [p[0] for p in pairs], [p[1] for p in pairs]
    assert len(set(dst)) == len(dst), f"two copies into one block: {pairs}"
    assert not set(src) & set(dst), f"a block is read and written by one list: {pairs}"


def test_private_blocks_of_a_full_pool_leave_sources_alone():
    """The one free block is taken; the first source, which only the prefix
    cache still names, must not become the second copy's destination."""
    alloc, cache, kv, s = cached_sequence(4, 40)
    named = s.block_table[:2]
    with pytest.raises(OutOfBlocksError):
        kv.make_private(s)
    pairs = kv.take_copies().tolist()
    check_pairs(pairs)
    assert pairs == [[named[0], s.block_table[0]]]
    kv.make_private(s)                           # that copy is on its way: its source can be evicted now
    check_pairs(kv.take_copies().tolist())
    assert not any(cache.holds(b) for b in s.block_table)


def test_sources_stay_cached_until_the_copies_are_taken():
    alloc, cache, kv, s = cached_sequence(6, 40)
    named = s.block_table[:2]
    kv.make_private(s)
    assert alloc.num_free == 1                   # the sources are not to be had yet
    other = [alloc.alloc()]
    with pytest.raises(OutOfBlocksError):
        alloc.alloc()
    n, blocks = cache.match(np.arange(40))       # but a lookup finds them
    assert n == 32 and blocks == named
    pairs = kv.take_copies().tolist()
    check_pairs(pairs)
    assert [p[0] for p in pairs] == named
    for b in blocks + other:
        alloc.decref(b)
    assert alloc.num_free == 3


def test_a_source_whose_last_holder_leaves_is_not_handed_out():
    """A fork copies a shared block; the other holder retires before the copy
    has run."""
    sc = Scheduler(BlockAllocator(3), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, 10, 4)
    b = sc.fork(a, 1, 4)
    x = a.block_table[0]
    sc.kv.slot_for(b, 10)
    sc.retire(a)
    check_invariants(sc)
    c = sc.restore(2, 10, 4)
    assert c.block_table != [x]
    check_invariants(sc)
    check_pairs(sc.kv.take_copies().tolist())
    assert sc.alloc.num_free == 1
    check_invariants(sc)


def test_a_copy_whose_destination_is_given_back_is_dropped():
    """make_private, truncate, make_private before the copies are taken: the
    block that comes back is the destination of one copy, not of two."""
    sc = Scheduler(BlockAllocator(5), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, 16, 4)
    x = sc.restore(1, 16, 4)
    b, y = sc.fork(a, 2, 4), sc.fork(x, 3, 4)
    free = sc.alloc.num_free
    sc.kv.make_private(b)
    sc.kv.truncate(b, 0)
    check_invariants(sc)
    assert sc.alloc.num_free == free and not sc.alloc.pins
    sc.kv.make_private(y)
    pairs = sc.kv.take_copies().tolist()
    check_pairs(pairs)
    assert pairs == [[x.block_table[0], y.block_table[0]]]
    check_invariants(sc)


def test_a_copy_whose_sequence_ends_is_dropped():
    sc = Scheduler(BlockAllocator(8), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, 40, 4)
    b = sc.fork(a, 1, 4)
    sc.kv.make_private(b, 20)
    sc.retire(b)
    sc.retire(a)
    assert sc.kv.take_copies().size == 0 and sc.alloc.num_free == 8 and sc.alloc.copies_emitted == 0
    check_invariants(sc)


def test_a_destination_that_others_still_hold_is_copied():
    """A destination that a fork holds, or that the prefix cache names, is not
    dropped with its first sequence, nor handed out again before its copy."""
    alloc, cache, kv, s = cached_sequence(5, 16)
    kv.make_private(s)
    t = kv.fork(s, 1, 4)
    (d,) = s.block_table
    kv.release(s)
    assert list(kv.pending_copies) == [d]
    cache.insert(np.arange(100, 116), [d])
    kv.release(t)
    for _ in range(3):
        assert alloc.alloc() != d
    with pytest.raises(OutOfBlocksError):        # the source and the destination wait for the copy
        alloc.alloc()
    check_pairs(kv.take_copies().tolist())
    n, blocks = cache.match(np.arange(100, 116))
    assert blocks == [d]


def test_a_copy_of_a_block_still_to_be_copied_comes_from_its_source():
    """A private copy is forked and copied again before the first copy ran."""
    sc = Scheduler(BlockAllocator(6), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, 16, 4)
    b = sc.fork(a, 1, 4)
    sc.kv.make_private(b)
    c = sc.fork(b, 2, 4)
    sc.kv.make_private(c)
    (x,), (y,), (z,) = a.block_table, b.block_table, c.block_table
    pairs = sc.kv.take_copies().tolist()
    check_pairs(pairs)
    assert pairs == [[x, y], [x, z]]
    check_invariants(sc)


def test_writing_behind_a_truncation_leaves_a_cached_block_alone():
    """A truncation can end inside a block that the prefix cache names; the
    next token goes into a copy, a later prompt still finds the original."""
    alloc, cache, kv, s = cached_sequence(8, 48)
    named = list(s.block_table)
    kv.truncate(s, 20)
    slot = kv.slot_for(s, 20)
    assert slot // 16 == s.block_table[1] != named[1] and slot % 16 == 4
    assert kv.take_copies().tolist() == [[named[1], s.block_table[1]]]
    n, blocks = cache.match(np.arange(48))
    assert n == 48 and blocks == named
    slot = kv.slot_for(s, 21)                    # its own now
    assert slot == s.block_table[1] * 16 + 5 and kv.take_copies().size == 0


def test_random_histories_keep_lists_pool_and_contents_sound():
    """Forks, private copies, truncations, retirements, appends and cached
    prefixes in any order, the copies run now and then, under a pool that is
    often full: every list can be copied at once, and every sequence's blocks
    hold its own tokens."""
    for seed in range(80):
        rng = np.random.default_rng(seed)
        sc = Scheduler(BlockAllocator(int(rng.integers(4, 24))), SchedulerConfig(watermark=0.0, prefix_cache=seed % 2 == 0))
        mem = np.full((sc.alloc.num_blocks, 16), -1)
        text, nxt, token = {}, 0, 0

        def run_copies():
            pairs = sc.kv.take_copies()
            check_pairs(pairs.tolist())
            if len(pairs):
                mem[pairs[:, 1]] = mem[pairs[:, 0]]

        for _ in range(200):
            op = rng.integers(0, 7)
            s = sc.running[int(rng.integers(0, len(sc.running)))] if sc.running else None
            try:
                if op == 0 or s is None:
                    n = int(rng.integers(1, 60))
                    if (n + 15) // 16 > sc.alloc.num_free:
                        continue
                    s = sc.restore(nxt, n, 4)
                    text[nxt] = list(range(token, token + n))
                    run_copies()
                    for i, t in enumerate(text[nxt]):
                        mem[s.block_table[i // 16], i % 16] = t
                    nxt, token = nxt + 1, token + n
                elif op == 1:
                    sc.fork(s, nxt, 4)
                    text[nxt] = list(text[s.seq_id])
                    nxt += 1
                elif op == 2:
                    sc.kv.make_private(s, int(rng.integers(0, 40)))
                elif op == 3:
                    n = int(rng.integers(0, s.num_cached + 1))
                    sc.kv.truncate(s, n)
                    del text[s.seq_id][n:]
                elif op == 4:
                    sc.retire(s)
                elif op == 5:
                    slot = sc.kv.slot_for(s, s.num_cached)
                    run_copies()
                    mem[slot // 16, slot % 16] = token
                    text[s.seq_id].append(token)
                    token += 1
                    s.num_cached += 1
                    s.prefill_end = s.num_cached
                elif sc.cache is not None:
                    sc.cache.insert(text[s.seq_id], s.block_table)
            except OutOfBlocksError:
                pass
            if rng.random() < 0.2:
                run_copies()
                for s in sc.running:
                    assert [mem[s.block_table[i // 16], i % 16] for i in range(s.num_cached)] == text[s.seq_id]
                if sc.cache is not None:
                    for s in sc.running:
                        n, blocks = sc.cache.match(text[s.seq_id])
                        got = [int(t) for x in blocks for t in mem[x]]
                        assert got == text[s.seq_id][:n]
                        for x in blocks:
                            sc.alloc.decref(x)
            check_invariants(sc)


def test_make_private_refuses_a_negative_position():
    """(It wrapped around to the sequence's last blocks.)"""
    sc = Scheduler(BlockAllocator(8), SchedulerConfig(watermark=0.0))
    b = sc.fork(sc.restore(0, 40, 4), 1, 4)
    with pytest.raises(ValueError):
        sc.kv.make_private(b, -1)
    assert sc.kv.take_copies().size == 0
