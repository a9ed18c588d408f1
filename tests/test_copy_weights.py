"""Block copies that take the attention weights along (pa_copy_blocks_weights):
a fork made private goes on with the sums its tokens had gathered."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import cache_ops_util as U
from paged_kv_cache_408_b200 import ops

FAKE, ODD = C.c_void_p(0x10000), C.c_void_p(0x10008)  # never dereferenced


def call(w=FAKE, n=3, k=FAKE, pairs=FAKE, d=128):
    return ops.lib().pa_copy_blocks_weights(k, FAKE, w, pairs, n, C.byref(ops.CacheDesc(64, 8, 16, d, 0)), None)


def test_refusals():
    assert call(w=None) == -1 and call(w=ODD) == -1 and call(k=None) == -1 and call(k=ODD) == -1 and call(pairs=None) == -1
    assert call(n=-1) == -1 and call(d=96) == -2
    assert call(n=0) == 0
    k, pairs = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.copy_blocks(k, k, pairs, weights=torch.zeros(4, 2, 16))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 128), (8, 128)])
def test_copies_are_bit_exact(cuda_device, Hkv, D, fp8):
    g = torch.Generator().manual_seed(Hkv + D)
    k, v = (torch.randint(0, 255, (40, Hkv, 16, D * (1 if fp8 else 2)), generator=g, dtype=torch.uint8) for _ in range(2))
    w = torch.randint(0, 1 << 31, (40, Hkv, 16), generator=g).int().view(torch.float32)
    perm = torch.randperm(40, generator=g)
    pairs = torch.stack([perm[:15], perm[15:30]], 1).int()
    as_cache = (lambda x: x.cuda()) if fp8 else (lambda x: x.cuda().view(torch.bfloat16))
    kd, vd, wd = as_cache(k), as_cache(v), w.cuda()
    ops.copy_blocks(kd, vd, pairs.cuda(), weights=wd)
    src, dst = pairs[:, 0].long(), pairs[:, 1].long()
    for x in (k, v, w.view(torch.int32)):
        x[dst] = x[src]
    assert torch.equal(kd.cpu().view(torch.uint8), k) and torch.equal(vd.cpu().view(torch.uint8), v)
    assert torch.equal(wd.cpu().view(torch.int32), w.view(torch.int32))
    with pytest.raises(ValueError):
        ops.copy_blocks(kd, vd, pairs.cuda(), weights=wd[:39])
    ops.copy_blocks(kd, vd, torch.tensor([[0, 40]], dtype=torch.int32).cuda(), weights=wd)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_PAIR


@pytest.mark.gpu
def test_a_fork_keeps_what_its_tokens_gathered(cuda_device):
    """Two decode steps with weights, a fork, private blocks (in which earlier
    owners left weights), two more steps of both, selection and compaction of
    the fork: its lists and sums are those of the whole history, and the other
    sequence's cache and sums keep their bits."""
    from paged_kv_cache_408_b200.runtime import BlockAllocator, Scheduler, SchedulerConfig, check_invariants
    Hkv, G, D, n, blocks, scale = 2, 4, 64, 90, 24, 0.125
    sc = Scheduler(BlockAllocator(blocks), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, n, 8)
    g = torch.Generator().manual_seed(17)
    k, v = (torch.randn(blocks, Hkv, 16, D, generator=g).bfloat16() for _ in range(2))
    qs = (torch.randn(4, 2, Hkv * G, D, generator=g) * 2).bfloat16()
    kd, vd = k.cuda(), v.cuda()
    w = (torch.rand(blocks, Hkv, 16, generator=g) * 50).cuda()       # what earlier owners left
    ws = ops.alloc_weights_workspace(2, Hkv * G, 6, kd)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()

    def step(i, tables, seen):
        q = qs[i, :len(tables)].cuda()
        ops.decode_weights(torch.empty_like(q), w, q, kd, vd, i32(tables), i32([n] * len(tables)), scale, ws,
                           i32(seen))

    step(0, [a.block_table], [0])
    step(1, [a.block_table], [n])
    b = sc.fork(a, 1, 8)
    sc.kv.make_private(b)
    ops.copy_blocks(kd, vd, torch.from_numpy(sc.kv.take_copies()).cuda(), weights=w)
    for i in (2, 3):
        step(i, [a.block_table, b.block_table], [n, n])
    t = np.arange(n)
    at = np.array(a.block_table)[t // 16], t % 16
    kept = w.cpu()[at[0], :, at[1]]                                   # a's sums, before b's are cut
    budget = 40
    keep, kl = torch.empty(1, Hkv, budget, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    ops.select_tokens(keep, kl, w, i32([b.block_table]), i32([n]), 4, 8)
    ops.compact_kv(kd, vd, i32([b.block_table]), keep, kl, w)
    sc.kv.compacted(b, budget)
    check_invariants(sc)
    sums = {0: torch.zeros(Hkv, n, dtype=torch.float64), 1: torch.zeros(Hkv, n, dtype=torch.float64)}
    slack = 0.0
    for i, row in [(0, 0), (1, 0), (2, 0), (3, 0), (0, 1), (1, 1), (2, 1), (3, 1)]:
        q = qs[i, row if i > 1 else 0]                                # the first two steps are both's
        for h in range(Hkv * G):
            _, p, _, dot = U.attend64(q[h].double(), k[at[0], h // G, at[1]].double(), v[at[0], h // G, at[1]].double(), scale,
                                      torch.ones(n, dtype=torch.bool))
            sums[row][h // G] += p
            slack = max(slack, U.score_slack(D, dot))
    tol = lambda x: (slack + 4 * (G + 1) * 2.0 ** -24) * x            # per weight, and the fp32 additions of 4 steps
    assert bool(((kept.double().T - sums[0]).abs() <= tol(sums[0])).all())
    out = keep[0].cpu().long()
    for h in range(Hkv):
        mine = sums[1][h]
        order = torch.sort(mine[4:n - 8], descending=True).values
        assert float(order[budget - 13] - order[budget - 12]) > 4 * float(tol(order[budget - 13]))  # (the cut is a clear one)
        want = sorted(list(range(4)) + [4 + int(x) for x in torch.topk(mine[4:n - 8], budget - 12).indices] + list(range(n - 8, n)))
        assert out[h].tolist() == want
        new = w.cpu()[np.array(b.block_table)[np.arange(budget) // 16], h, np.arange(budget) % 16].double()
        assert bool(((new - mine[out[h]]).abs() <= tol(mine[out[h]])).all())
    assert U.same_bits(kd[a.block_table], k[a.block_table]) and U.same_bits(vd[a.block_table], v[a.block_table])
    assert U.same_bits(w.cpu()[at[0], :, at[1]], kept)
    assert ops.get_last_device_error() == 0
