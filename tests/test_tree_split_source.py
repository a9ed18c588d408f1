"""The split of tree attention over CTAs, as the kernel's own source computes
it (csrc/tree_split.h compiled for the host): every key tile of every segment
in exactly one share, no slot for partial results used twice, the pieces that
the merge expects the ones written, and the shares balanced."""
import ctypes as C
import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("tree_split") / "split.so")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "paged_kv_cache_408_b200", "csrc"),
                    "-isystem", cuda, os.path.join(HERE, "tree_split_host.cpp"), "-o", so], check=True)
    lib = C.CDLL(so)

    def items(seqs, heads, G, e4m3, ctas, max_blocks=None, max_q=64, cu=None):
        """seqs: (drafts, prefix) -> rows (CTA, sequence, kv head, first draft, row tiles, j0, j1, tiles, slot, pieces)."""
        cu = np.concatenate([[0], np.cumsum([d for d, _ in seqs])]).astype(np.int32) if cu is None else np.array(cu, np.int32)
        prefix = np.array([p for _, p in seqs], np.int32)
        room = 4 * heads * len(seqs) + 4 * ctas
        out = np.zeros((room, 10), np.int32)
        blocks = max_blocks or max(-(-(d + p) // 16) for d, p in seqs) + 1
        n = lib.tree_items(cu.ctypes.data_as(C.c_void_p), prefix.ctypes.data_as(C.c_void_p), len(seqs), blocks, heads, G,
                           max_q, int(cu[-1]), int(e4m3), ctas, out.ctypes.data_as(C.c_void_p), room)
        assert n >= 0
        return out[:n].tolist()

    return items, lib.tree_piece_slot_of


def expected_tiles(seqs, heads, G):
    """{(sequence, kv head, first draft): (row tiles, key tiles)}"""
    want = {}
    for b, (drafts, prefix) in enumerate(seqs):
        tiles = -(-drafts * G // 128)
        for r in range(0, tiles, 2):
            for h in range(heads):
                want[b, h, r * (128 // G)] = (min(2, tiles - r), -(-(drafts + prefix) // 128))
    return want


def check(split, seqs, heads, G, e4m3, ctas):
    items, piece_slot = split
    rows = items(seqs, heads, G, e4m3, ctas)
    want = expected_tiles(seqs, heads, G)
    got, slots, cut = {}, {}, {}
    for cta, b, h, r0, rt, j0, j1, nt, slot, pieces in rows:
        key = (b, h, r0)
        assert 0 <= j0 < j1 <= nt and want[key] == (rt, nt)
        for j in range(j0, j1):
            assert (key, j) not in got
            got[key, j] = cta
        if slot >= 0:
            assert slot not in slots and slot // 2 == cta
            slots[slot] = key
        if pieces:
            assert slot >= 0 and cta not in cut
            cut[cta] = (key, pieces)
    assert len(got) == sum(nt for _, nt in want.values())
    used = set()
    for cta, (key, pieces) in cut.items():
        for p in range(pieces):
            slot = piece_slot(cta, p)
            assert slots.get(slot) == key
            used.add(slot)
    assert used == set(slots)
    return got, rows


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_tile_once_and_every_piece_merged(split, e4m3):
    for seed in range(250):
        rnd = random.Random(seed)
        seqs = [(rnd.choice([0, 1, 16, 33, 64, rnd.randint(0, 64)]), rnd.choice([0, 1, 127, 128, rnd.randint(0, 3000)]))
                for _ in range(rnd.randint(1, 20))]
        check(split, seqs, rnd.choice([1, 2, 3, 8]), rnd.choice([1, 2, 4, 8]), e4m3, rnd.choice([1, 2, 7, 148]))


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_and_many(split, e4m3):
    check(split, [(64, 300000)], 8, 8, e4m3, 148)
    rnd = random.Random(1)
    check(split, [(rnd.randint(0, 3), rnd.randint(0, 40)) for _ in range(2048)], 2, 2, e4m3, 148)


def test_sequences_with_bad_lengths_take_no_share(split):
    items, _ = split
    rows = items([(4, 40), (4, 10 ** 6), (4, -1), (5, 60), (4, 0)], 2, 2, False, 148, max_blocks=8, max_q=4)
    assert {r[1] for r in rows} == {0, 4}
    rows = items([(4, 40), (4, 50), (4, 60)], 2, 2, False, 148, cu=[0, 8, 4, 12], max_blocks=8, max_q=8)
    assert {r[1] for r in rows} == {0, 2}        # the second one's rows run backwards


def test_shares_are_balanced(split):
    """64 sequences of U[1, 2048] tokens, 16 drafts, 8 kv heads of 4: no CTA
    has more than one segment's start and a tile above the mean."""
    seqs = [(16, 1 + (2 * i + 1) * 16) for i in range(64)]
    got, rows = check(split, seqs, 8, 4, False, 148)
    cost = [0] * 148
    for cta, _, _, _, _, j0, j1, *_ in rows:
        cost[cta] += 2 * (j1 - j0) + 5
    assert min(cost) > 0 and max(cost) <= sum(cost) / 148 + 2 * 5 + 2
