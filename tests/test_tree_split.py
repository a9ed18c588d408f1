"""The split of tree attention over CTAs, restated on the host: the segments
(sequence, kv head, one or two row tiles) form one line of cost units that is
cut into equal shares; every key tile belongs to exactly one share, the two
slots a CTA has for partial results are never used twice, and the pieces that
the merge kernel expects of a cut segment are the ones written."""
import random

import pytest

ONE, PAIR = 2, 3  # units of a key tile with one and with two row tiles


def split(seqs, heads, qpos, seg_cost, ctas):
    """seqs: (drafts, prefix) -> {(b, head, segment, tile): CTA}, slots, merges."""
    rows = []
    for drafts, prefix in seqs:
        tiles = -(-drafts // qpos)
        nt = -(-(prefix + drafts) // 128) if drafts else 0
        npair, none = tiles >> 1, tiles & 1
        rows.append((npair, none, nt, npair * (seg_cost + nt * PAIR) + none * (seg_cost + nt * ONE)))
    total = sum(r[3] * heads for r in rows)
    S = max(-(-total // ctas), PAIR)
    owner, slots, merges = {}, {}, {}
    for g in range(ctas):
        pos = min(g * S, total)
        end, base, b = min(pos + S, total), 0, 0
        while pos < end and pos >= base + rows[b][3] * heads:
            base, b = base + rows[b][3] * heads, b + 1
        while pos < end:
            npair, none, nt, head = rows[b]
            off = pos - base
            if off >= head * heads:
                base, b = base + head * heads, b + 1
                continue
            kvh, r = divmod(off, head)
            seg = min(r // (seg_cost + nt * PAIR), npair)
            r -= seg * (seg_cost + nt * PAIR)
            unit = PAIR if seg < npair else ONE
            stop = min(seg_cost + nt * unit, end - pos + r)
            j0, j1 = (max(0, x - seg_cost + unit - 1) // unit for x in (r, stop))
            start = pos - r
            pos = start + stop
            if j1 <= j0:
                continue
            key = (b, kvh, seg)
            for j in range(j0, j1):
                assert key + (j,) not in owner
                owner[key + (j,)] = g
            if (j0, j1) != (0, nt):
                slot = 2 * g + (j0 == 0)
                assert slot not in slots
                slots[slot] = key
                if j0 == 0:
                    assert pos >= end  # the share's last
                    first = start + seg_cost
                    merges[g] = (key, (first + (nt - 1) * unit) // S - first // S + 1)
    return owner, slots, merges, sum(heads * (p + o) * nt for p, o, nt, _ in rows)


@pytest.mark.parametrize("seg_cost", [5, 7])
def test_every_tile_once_and_every_piece_merged(seg_cost):
    for seed in range(600):
        rnd = random.Random(seed)
        seqs = [(rnd.choice([0, 1, 16, 33, 64, rnd.randint(0, 64)]), rnd.choice([0, 1, 127, 128, rnd.randint(0, 3000)]))
                for _ in range(rnd.randint(1, 20))]
        owner, slots, merges, tiles = split(seqs, rnd.choice([1, 2, 3, 8]), 128 // rnd.choice([1, 2, 4, 8]), seg_cost,
                                            rnd.choice([1, 2, 7, 148]))
        assert len(owner) == tiles
        used = set()
        for g, (key, pieces) in merges.items():
            for p in range(pieces):
                slot = 2 * (g + p) + (p == 0)
                assert slots.get(slot) == key
                used.add(slot)
        assert used == set(slots)


def test_shares_are_balanced():
    """64 sequences of U[1, 2048] tokens, 16 drafts, 8 kv heads: no CTA gets
    more than one tile above the others' share of the line."""
    seqs = [(16, 1 + (2 * i + 1) * 16) for i in range(64)]
    owner, _, _, tiles = split(seqs, 8, 32, 5, 148)
    per = {}
    for key, g in owner.items():
        per.setdefault(g, []).append(key)
    cost = [len(k) * ONE + 5 * len({x[:3] for x in k}) for k in per.values()]
    assert max(cost) <= sum(cost) / len(cost) + 2 * 5 + ONE
