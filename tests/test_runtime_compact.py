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


def prompt_sequence(sc, seq_id, n, decode_left=20):
    s = Sequence(seq_id, n, decode_left, tokens=np.arange(n) + 1000 * seq_id)
    sc.add_request(s)
    while s.status != "running" or s.in_prefill:
        sc.complete(sc.step())
    return s


def cut(sc, s, n):
    """make_private, (selection, compaction,) release of what is behind."""
    sc.kv.make_private(s)
    sc.kv.take_copies()
    sc.kv.compacted(s, n)
    check_invariants(sc)


def test_a_compacted_sequence_that_is_preempted_recomputes_its_whole_text():
    """Its kept tokens are no beginning of its text: it comes back with all of
    them, cached prefixes found by the prompt's own tokens."""
    sc = scheduler(blocks=20, prefix_cache=True)
    s = prompt_sequence(sc, 0, 100)
    named = list(s.block_table[:6])
    cut(sc, s, 32)
    assert s.num_cached == 32 and s.num_dropped == 68 and len(s.block_table) == 2 and s.num_tokens == 101
    sc.complete(sc.step())                       # one token behind the kept ones
    assert s.num_cached == 33 and s.num_tokens == 102
    plan = sc.step()
    assert sc._preempt_one(plan, s) is s
    assert s.prefill_end == 101 and s.num_cached == 0 and s.num_dropped == 0  # the prompt and the token decoded
    sc._inflight = ([], [])
    while s.in_prefill or s.status != "running":
        plan = sc.step()
        if 0 in plan.prefill_ids.tolist():
            at = plan.prefill_ids.tolist().index(0)
            assert plan.prefill_prefix[at] == 96 and plan.prefill_tables[at, :6].tolist() == named
        sc.complete(plan)
    assert s.num_cached == 101 and len(s.block_table) == 7 and s.num_tokens == 102
    check_invariants(sc)


def test_a_fork_of_a_compacted_sequence_knows_what_it_lacks():
    sc = scheduler()
    s = prompt_sequence(sc, 0, 60)
    cut(sc, s, 20)
    f = sc.fork(s, 1, 4)
    assert f.num_dropped == 40 and f.num_tokens == 61
    with pytest.raises(ValueError):
        sc.kv.compacted(s, 21)                   # more than it holds
    sc.kv.truncate(f, 18)                        # two tokens back
    assert f.num_tokens == 59 and f.num_dropped == 40


def test_a_sequence_compacted_while_its_prompt_is_read():
    """The rest of the prompt is still read, and what remains is not cached
    under the prompt's tokens."""
    sc = scheduler(blocks=32, prefix_cache=True, max_num_batched_tokens=40, max_chunk=40)
    s = Sequence(0, 100, 4, tokens=np.arange(100))
    sc.add_request(s)
    sc.complete(sc.step())
    assert s.num_cached == 40 and s.in_prefill
    cut(sc, s, 16)
    read = 40
    while s.in_prefill:
        plan = sc.step()
        read += plan.num_prefill_tokens
        sc.complete(plan)
    assert read == 100 and s.num_cached == 76 and s.num_tokens == 101
    assert sc.cache.peek(np.arange(100)) == 0
    check_invariants(sc)


def test_a_compacted_text_that_outgrew_its_table_is_not_preempted():
    """Two sequences of more text than a table holds, kept in it by
    compaction: neither can be recomputed, so neither is evicted; the step
    that could only evict one says so."""
    sc = scheduler(blocks=6, max_blocks_per_seq=4)
    a, b = sc.restore(0, 40, 100), sc.restore(1, 40, 100)
    for _ in range(3):
        for _ in range(8):
            sc.complete(sc.step())
        cut(sc, a, 40)
        cut(sc, b, 40)
    assert a.num_dropped == b.num_dropped == 24 and not sc.num_preemptions
    assert sc.alloc.free_list == []               # three blocks each
    for _ in range(8):
        sc.complete(sc.step())
    with pytest.raises(OutOfBlocksError):
        sc.step()
    assert sc.num_preemptions == 0 and [s.seq_id for s in sc.running] == [0, 1]
    check_invariants(sc)
    cut(sc, a, 20)
    plan = sc.step()                              # there is room again
    assert plan.decode_ids.tolist() == [0, 1]


def test_the_youngest_that_can_be_recomputed_gives_way():
    """A sequence whose slot of this step is given is not evicted for a later
    one that cannot give way itself."""
    sc = scheduler(blocks=6, max_blocks_per_seq=4)
    a, b = prompt_sequence(sc, 0, 30), prompt_sequence(sc, 1, 60, 100)
    cut(sc, b, 48)
    sc.kv.truncate(b, 48)
    b.num_dropped = 30                            # a text of 78 tokens, more than 4 blocks
    sc.complete(sc.step())                        # b takes the fourth block of its table, the pool's last
    assert sc.alloc.free_list == []
    while len(a.block_table) * 16 > a.num_cached:
        sc.complete(sc.step())
    plan = sc.step()                              # a needs a block: it gives way, the younger b cannot
    assert plan.preempted == [0] and plan.decode_ids.tolist() == [1]
    check_invariants(sc)
