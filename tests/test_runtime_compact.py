"""Block bookkeeping of drafts and of compacted sequences: private blocks
before an in-place move, blocks behind a truncation given back."""
import numpy as np
import pytest

from paged_kv_cache_408_b200.runtime import (BlockAllocator, KVManager, OutOfBlocksError, PrefixCache, Scheduler,
                                             SchedulerConfig, Sequence, check_invariants)


def scheduler(blocks=32, **kw):
    return Scheduler(BlockAllocator(blocks), SchedulerConfig(watermark=0.0, **kw))


def test_truncate_releases_whole_blocks_only():
    sc = scheduler()
    s = sc.restore(0, 50, 4)                     # 4 blocks
    free = sc.alloc.num_free
    sc.kv.truncate(s, 33)                        # the third block keeps one position
    assert len(s.block_table) == 3 and s.num_cached == 33 and sc.alloc.num_free == free + 1
    assert not s.in_prefill and s.num_tokens == 34
    sc.kv.truncate(s, 32)
    assert len(s.block_table) == 2
    check_invariants(sc)
    plan = sc.step()                             # the next token opens a new block
    assert plan.decode_lens.tolist() == [33] and len(s.block_table) == 3
    sc.complete(plan)
    sc.kv.truncate(s, 0)
    assert s.block_table == [] and s.num_cached == 0
    check_invariants(sc)
    with pytest.raises(ValueError):
        sc.kv.truncate(s, 1)
    with pytest.raises(ValueError):
        sc.kv.truncate(s, -1)


def test_drafts_are_slots_behind_the_cached_tokens():
    sc = scheduler()
    s = sc.restore(0, 30, 4)
    slots = [sc.kv.slot_for(s, 30 + i) for i in range(5)]
    assert [x % 16 for x in slots] == [14, 15, 0, 1, 2] and len(s.block_table) == 3
    sc.kv.truncate(s, 31)                        # one draft accepted
    assert len(s.block_table) == 2 and s.num_cached == 31
    check_invariants(sc)


def test_make_private_copies_shared_blocks_from_a_position_on():
    sc = scheduler()
    a = sc.restore(0, 50, 4)
    b = sc.fork(a, 1, 4)
    before = list(a.block_table)
    sc.kv.make_private(b, 20)                    # block 0 stays shared
    copies = sc.kv.take_copies()
    assert b.block_table[0] == before[0] and a.block_table == before
    assert copies.tolist() == [[before[j], b.block_table[j]] for j in (1, 2, 3)]
    assert len(set(b.block_table[1:]) & set(before)) == 0
    check_invariants(sc)
    sc.kv.make_private(b, 20)                    # its own already
    assert sc.kv.take_copies().size == 0
    sc.kv.truncate(b, 17)
    sc.retire(a)
    sc.kv.make_private(b)                        # no longer shared
    assert sc.kv.take_copies().size == 0
    check_invariants(sc)


def test_make_private_leaves_cached_prefixes_alone():
    """A block that the prefix cache names keeps its contents: the sequence
    goes on with a copy, a later prompt still finds the original."""
    alloc = BlockAllocator(16)
    cache = PrefixCache(alloc)
    kv = KVManager(alloc)
    s = Sequence(0, 40, 4, 40, 40, False, [alloc.alloc() for _ in range(3)])
    tokens = np.arange(40)
    cache.insert(tokens, s.block_table)
    named = s.block_table[:2]
    kv.make_private(s)
    assert not set(named) & set(s.block_table) and len(kv.take_copies()) == 2
    n, blocks = cache.match(tokens)
    assert n == 32 and blocks == named


def test_make_private_out_of_blocks():
    sc = scheduler(blocks=5)
    a = sc.restore(0, 48, 4)
    b = sc.fork(a, 1, 4)
    with pytest.raises(OutOfBlocksError):
        sc.kv.make_private(b)
    check_invariants(sc)                         # what was copied is consistent
    assert len(sc.kv.take_copies()) == 2
