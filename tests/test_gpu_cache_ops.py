"""GPU tests of the calls that serve drafts and cache budgets: tree attention
(pa_decode_tree), decode with attention weights (pa_decode_weights), token
selection (pa_select_tokens) and compaction (pa_compact_kv), each against a
plain form in 64 bits (cache_ops_util)."""
import math

import numpy as np
import pytest
import torch

import cache_ops_util as U
from paged_kv_cache_408_b200 import ops

pytestmark = pytest.mark.gpu


def dev(x):
    return None if x is None else x.cuda()


def run_tree(c, q, cu, prefix, mask, scale, max_q=None, fill=7.0, pad_rows=0):
    """Output on the host; the workspace starts as 0xFF bytes; `pad_rows` rows
    behind the last sequence."""
    sizes = [cu[i + 1] - cu[i] for i in range(len(cu) - 1)]
    max_q = max(sizes) if max_q is None else max_q
    if pad_rows:
        q = torch.cat([q, torch.ones(pad_rows, *q.shape[1:], dtype=q.dtype)])
        mask = torch.cat([mask, torch.full((pad_rows,), -1, dtype=torch.int64)])
    qd, kd = dev(q), dev(c.k)
    out = torch.full_like(qd, fill)
    ws = ops.alloc_tree_workspace(len(prefix), q.shape[1], max_q, c.tables.shape[1], kd)
    ws.fill_(0xFF)
    ops.decode_tree(out, qd, torch.tensor(cu, dtype=torch.int32).cuda(),
                    torch.tensor(prefix, dtype=torch.int32).cuda(), dev(mask), dev(c.tables), kd, dev(c.v), scale,
                    max_q, ws, dev(c.k_scale), dev(c.v_scale))
    torch.cuda.synchronize()
    return out.cpu()


def check_tree(c, q, cu, prefix, mask, scale, **kw):
    total = q.shape[0]
    out = run_tree(c, q, cu, prefix, mask, scale, **kw)
    assert ops.get_last_device_error() == 0
    ref, tol = U.tree64(c, q, cu, prefix, mask, scale, 2.0 ** -11 if c.k_scale is not None else 2.0 ** -8)
    err = (out[:total].double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err - tol).max()):.3e} beyond the tolerance"
    assert bool((out[total:] == 7.0).all()), "rows behind the last sequence were written"


def make_tree(seed, prefix, sizes, Hkv, G, D, fp8=False, qmul=1.5):
    c = U.paged(seed, [p + t for p, t in zip(prefix, sizes)], Hkv, D, fp8)
    cu = [0] + list(np.cumsum(sizes).tolist())
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(cu[-1], Hkv * G, D, generator=g) * qmul).bfloat16()
    return c, q, cu, list(prefix), U.tree_masks(seed + 2, sizes), 1 / math.sqrt(D)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_shapes(cuda_device, D, G, fp8):
    """Prefixes that end on, before and behind blocks and key tiles, trees of 1 to 64 drafts, none and no prefix."""
    prefix = [0, 1, 15, 16, 40, 127, 128, 129, 300, 64, 0, 33]
    sizes = [5, 64, 1, 16, 33, 1, 7, 64, 31, 0, 1, 17]
    check_tree(*make_tree(D + G, prefix, sizes, 2, G, D, fp8), pad_rows=3)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_one_long_sequence(cuda_device, fp8):
    """A long prefix over few heads: every row is split into many pieces."""
    check_tree(*make_tree(3, [9001], [9], 1, 4, 128, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_many_sequences(cuda_device, fp8):
    """More rows than the GPU holds at once, of all lengths."""
    rng = np.random.RandomState(4)
    prefix, sizes = rng.randint(0, 200, 150).tolist(), rng.randint(0, 20, 150).tolist()
    check_tree(*make_tree(4, prefix, sizes, 3, 2, 64, fp8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_masks(cuda_device, D, fp8):
    """Rows that see nothing (zeros), everything, only others, bits past the last draft."""
    c, q, cu, prefix, _, scale = make_tree(5, [0, 0, 130, 3], [8, 64, 8, 1], 2, 4, D, fp8)
    rows = [0, -1, 1 << 7, 0, (1 << 8), 3, 1 << 63, 0xF0] + [(-1 if i % 3 else 1 << (63 - i)) for i in range(64)] + \
        [0, -1, 1, 2, 4, 1 << 20, 0, 0x55] + [1 << 1]
    mask = torch.tensor([r - (1 << 64) if r >= 1 << 63 else r for r in rows], dtype=torch.int64)
    check_tree(c, q, cu, prefix, mask, scale)
    out = run_tree(c, q, cu, prefix, mask, scale)
    assert bool((out[0] == 0).all()) and bool((out[3] == 0).all()) and bool((out[4] == 0).all())


@pytest.mark.parametrize("qmul", [1e-3, 40.0])
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_score_ranges(cuda_device, fp8, qmul):
    """Nearly uniform and nearly one-hot softmaxes."""
    check_tree(*make_tree(6, [500, 77], [20, 3], 2, 2, 128, fp8, qmul))


def test_tree_growing_scores(cuda_device):
    """Scores that grow along the sequence move the running maximum at every tile."""
    c, q, cu, prefix, mask, scale = make_tree(7, [1500], [12], 1, 4, 128)
    t = torch.arange(1512)
    grow = (0.02 + t.float() / 300)[:, None]
    blk = c.tables[0].long()[t // 16]
    c.k[blk, 0, t % 16] = (q[0, 0].float()[None] * grow + 0.1 * c.k[blk, 0, t % 16].float()).bfloat16()
    check_tree(c, q, cu, prefix, mask, scale)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("prefix", [0, 100, 1000])
def test_tree_masked_nonfinite_drafts(cuda_device, prefix, bad, fp8):
    """NaN and infinities in the K and V of drafts that a row does not see stay out of its output."""
    if fp8 and math.isinf(bad):
        pytest.skip("E4M3 has no infinities")
    c, q, cu, pre, _, scale = make_tree(8, [prefix, 20], [12, 4], 2, 4, 128, fp8)
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(12)] + [1, 2, 4, 8], dtype=torch.int64)
    for j in (5, 9):  # rows 0..4 see neither
        t = prefix + j
        for x, cols in ((c.k, slice(3, 5)), (c.v, slice(0, 128, 7))):
            x.view(torch.uint8 if fp8 else torch.int16)[int(c.tables[0, t // 16]), :, t % 16, cols] = \
                torch.tensor(bad).to(c.k.dtype).view(torch.uint8 if fp8 else torch.int16)
    out = run_tree(c, q, cu, pre, mask, scale)
    ref, tol = U.tree64(c, q, cu, pre, mask, scale, 2.0 ** -8)
    ok = torch.tensor([True] * 5 + [False] * 7 + [True] * 4)
    err = (out.double() - ref).abs()
    assert bool((err[ok] <= tol[ok]).all())


def test_tree_visible_nonfinite_value(cuda_device):
    """A visible draft's infinite or NaN V element reaches exactly the rows and columns that see it."""
    c, q, cu, pre, _, scale = make_tree(9, [70], [6], 1, 2, 64)
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(6)], dtype=torch.int64)
    t = 70 + 3
    c.v[int(c.tables[0, t // 16]), 0, t % 16, 5] = math.inf
    c.v[int(c.tables[0, t // 16]), 0, t % 16, 9] = math.nan
    out = run_tree(c, q, cu, pre, mask, scale).double()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[3:, :, 5] = True
    bad[3:, :, 9] = True
    assert bool(torch.isfinite(out[~bad]).all())
    assert bool((out[3:, :, 5] == math.inf).all()) and bool(torch.isnan(out[3:, :, 9]).all())
    ref, tol = U.tree64(c, q, cu, pre, mask, scale, 2.0 ** -8)
    assert bool(((out - ref).abs()[~bad] <= tol[~bad]).all())


def test_tree_bad_metadata(cuda_device):
    """Bad lengths leave a sequence's rows as they are, a bad block is flagged and the rest computed."""
    c, q, cu, pre, mask, scale = make_tree(10, [40, 50, 60], [4, 4, 4], 2, 2, 64)
    ops.get_last_device_error()
    out = run_tree(c, q, cu, [40, 10 ** 6, 60], mask, scale)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN
    ref, tol = U.tree64(c, q, cu, pre, mask, scale, 2.0 ** -8)
    err = (out.double() - ref).abs()
    assert bool((err[:4] <= tol[:4]).all()) and bool((err[8:] <= tol[8:]).all()) and bool((out[4:8] == 7).all())
    out = run_tree(c, q, cu, [40, -1, 60], mask, scale)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN and bool((out[4:8] == 7).all())
    with pytest.raises(ops.PAError):  # 12 rows, at most 3 x 3
        run_tree(c, q, cu, pre, mask, scale, max_q=3)
    out = run_tree(c, q, [0, 2, 7, 12], pre, mask, scale, max_q=4)  # 5 drafts where at most 4 were announced
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN and bool((out[2:] == 7).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_bad_block(cuda_device, D, fp8):
    """A bad table entry is flagged and its keys are absent, as if they were not there."""
    c, q, cu, pre, mask, scale = make_tree(11, [400, 50], [4, 4], 2, 2, D, fp8)
    bad = [5, 24]                                    # prefix tokens 80..95, 384..399
    c.tables[0, bad[0]], c.tables[0, bad[1]] = 10 ** 6, -1
    ops.get_last_device_error()
    out = run_tree(c, q, cu, pre, mask, scale)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_BLOCK
    ok = U.Paged(c.k, c.v, c.tables.clamp(0, c.k.shape[0] - 1), c.k_scale, c.v_scale)
    ref, tol = U.tree64(ok, q, cu, pre, mask, scale, 2.0 ** -8)
    assert bool(((out.double() - ref).abs()[4:] <= tol[4:]).all())
    k, v = ok.rows64("k", 0, 404), ok.rows64("v", 0, 404)
    for i in range(4):
        see = torch.tensor([t // 16 not in bad for t in range(400)] + [bool((int(mask[i]) >> j) & 1) for j in range(4)])
        for h in range(4):
            o, _, av, dot = U.attend64(q[i, h].double(), k[:, h // 2], v[:, h // 2], scale, see)
            assert bool(((out[i, h].double() - o).abs() <=
                         2.0 ** -8 * o.abs() + (2.0 ** -8 + U.score_slack(D, dot)) * av).all())


def test_tree_most_sequences(cuda_device):
    """2048 sequences, most of them without drafts."""
    rng = np.random.RandomState(15)
    sizes = (rng.randint(0, 6, 2048) // 5 * rng.randint(1, 4, 2048)).tolist()
    check_tree(*make_tree(15, rng.randint(0, 30, 2048).tolist(), sizes, 1, 2, 64))


def test_tree_no_drafts_at_all(cuda_device):
    """Rows behind the last sequence only: nothing is written."""
    c, q, cu, pre, mask, scale = make_tree(16, [20, 3], [0, 0], 1, 2, 64)
    out = run_tree(c, q, cu, pre, mask, scale, max_q=2, pad_rows=3)
    assert bool((out == 7.0).all()) and ops.get_last_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 8])
def test_tree_smallest(cuda_device, G, fp8):
    """One draft of one sequence (fewer rows than a copy box), with and without a prefix."""
    for prefix in (0, 1, 130):
        check_tree(*make_tree(12 + prefix, [prefix], [1], 1, G, 64, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_many_long_segments(cuda_device, fp8):
    """Segments cut at every place: two row tiles, one, and both in a sequence."""
    check_tree(*make_tree(13, [3000, 700, 5, 1290, 2048], [64, 17, 33, 48, 16], 2, 8, 64, fp8))


def test_calls_refuse_another_current_device(cuda_device, monkeypatch):
    c, q, cu, pre, mask, scale = make_tree(14, [40], [4], 2, 2, 64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        run_tree(c, q, cu, pre, mask, scale)


# --------------------------------------------------------- attention weights
def run_weights(c, q, lens, scale, w, seen):
    qd, kd = dev(q), dev(c.k)
    out, wd = torch.full_like(qd, 7.0), dev(w).clone()
    ws = ops.alloc_weights_workspace(q.shape[0], q.shape[1], c.tables.shape[1], kd)
    ws.fill_(0xFF)
    ops.decode_weights(out, wd, qd, kd, dev(c.v), dev(c.tables), torch.tensor(lens, dtype=torch.int32).cuda(), scale,
                       ws, None if seen is None else torch.tensor(seen, dtype=torch.int32).cuda(), dev(c.k_scale),
                       dev(c.v_scale))
    torch.cuda.synchronize()
    return out.cpu(), wd.cpu()


def check_weights(seed, lens, Hkv, G, D, fp8=False, seen=None, qmul=1.5):
    c = U.paged(seed, lens, Hkv, D, fp8)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), Hkv * G, D, generator=g) * qmul).bfloat16()
    w = torch.rand(c.k.shape[:3], generator=g) * 3
    old = [n - 1 for n in lens] if seen is None else seen
    for b, n in enumerate(lens):  # what nobody has written yet
        for t in range(max(0, old[b]), n):
            w[int(c.tables[b, t // 16]), :, t % 16] = math.nan
    out, wd = run_weights(c, q, lens, 1 / math.sqrt(D), w, old)
    assert ops.get_last_device_error() == 0
    ref, tol, wr, wtol = U.weights64(c, q, lens, 1 / math.sqrt(D), w, old)
    assert bool(((out.double() - ref).abs() <= tol).all())
    touched = wtol > 0
    assert U.same_bits(wd[~touched], w[~touched]), "a slot of no cached token was written"
    assert bool(((wd.double() - wr).abs()[touched] <= wtol[touched]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_shapes(cuda_device, D, G, fp8):
    check_weights(D + G, [1, 0, 15, 16, 17, 100, 700, 33, 256, 257], 2, G, D, fp8)


@pytest.mark.parametrize("fp8,G", [(False, 4), (True, 8), (True, 2)])
def test_weights_long(cuda_device, fp8, G):
    check_weights(21, [9003, 40], 1, G, 128, fp8)


def test_weights_first_step(cuda_device):
    """seen 0: every slot starts at zero, whatever it held."""
    check_weights(22, [50, 3, 0], 2, 4, 64, seen=[0, 0, 0])


def test_weights_all_seen(cuda_device):
    check_weights(23, [50, 3], 2, 4, 64, seen=[50, 1000])


@pytest.mark.parametrize("qmul", [1e-3, 40.0])
def test_weights_score_ranges(cuda_device, qmul):
    check_weights(24, [600, 31], 2, 4, 128, qmul=qmul)


def test_weights_many(cuda_device):
    rng = np.random.RandomState(25)
    check_weights(25, rng.randint(0, 150, 200).tolist(), 3, 2, 64)


def test_weights_seen_none_adds_to_all(cuda_device):
    c = U.paged(26, [40, 9], 2, 64)
    q = torch.randn(2, 4, 64).bfloat16()
    w = torch.rand(c.k.shape[:3])
    _, a = run_weights(c, q, [40, 9], 0.125, w, None)
    _, b = run_weights(c, q, [40, 9], 0.125, w, [40, 9])
    assert U.same_bits(a, b)


def test_weights_bad_metadata(cuda_device):
    c = U.paged(27, [40, 9], 2, 64)
    q = torch.randn(2, 4, 64).bfloat16()
    w = torch.rand(c.k.shape[:3])
    ops.get_last_device_error()
    _, a = run_weights(c, q, [40, 10 ** 6], 0.125, w, [0, 0])
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN
    _, b = run_weights(c, q, [40, 0], 0.125, w, [0, 0])
    assert ops.get_last_device_error() == 0 and U.same_bits(a, b)
    c.tables[0, 1] = -1
    _, a = run_weights(c, q, [40, 9], 0.125, w, [0, 0])
    assert ops.get_last_device_error() == ops.DEVERR_BAD_BLOCK


@pytest.mark.parametrize("fp8,G", [(False, 4), (True, 2), (True, 8)])
@pytest.mark.parametrize("n", [40, 3000])
def test_weights_nan_key(cuda_device, fp8, G, n):
    """A NaN in a key makes every weight of its sequence and kv head NaN, as
    the softmax over it is, in one piece or in many; no other weight."""
    c = U.paged(28, [n, n], 2, 64, fp8)
    t = n // 2
    c.k.view(torch.uint8 if fp8 else torch.int16)[int(c.tables[0, t // 16]), 1, t % 16, 3] = 0x7f if fp8 else 0x7fc0
    q = torch.randn(2, 2 * G, 64).bfloat16()
    out, w = run_weights(c, q, [n, n], 0.125, torch.zeros(c.k.shape[:3]), [0, 0])
    tok = torch.arange(n)
    for b in range(2):
        for h in range(2):
            bad = b == 0 and h == 1
            assert bool((torch.isnan(w[c.tables[b].long()[tok // 16], h, tok % 16]) == bad).all())
            assert bool((torch.isnan(out[b, h * G:(h + 1) * G]) == bad).all())


# ------------------------------------------------------------------ selection
def check_select(seed, lens, Hkv, budget, sink, recent, make=None, width=None):
    rng = np.random.RandomState(seed)
    nb = [(n + 15) // 16 for n in lens]
    pool = sum(nb) + 2
    perm = rng.permutation(pool)
    tables = np.full((len(lens), width or max(max(nb), 1)), -1, np.int32)
    at = 0
    for b in range(len(lens)):
        tables[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    w = (rng.rand(pool, Hkv, 16) ** 6 * 3).astype(np.float32)
    w[w < 1e-3] = 0
    if make:
        make(w, rng)
    keep = torch.full((len(lens), Hkv, budget), 77, dtype=torch.int32, device="cuda")
    kl = torch.full((len(lens),), 77, dtype=torch.int32, device="cuda")
    ops.select_tokens(keep, kl, torch.from_numpy(w).cuda(), torch.from_numpy(tables).cuda(),
                      torch.tensor(lens, dtype=torch.int32).cuda(), sink, recent)
    assert ops.get_last_device_error() == 0
    ref, got = U.select_plain(w, tables, lens, budget, sink, recent)
    assert np.array_equal(kl.cpu().numpy(), got)
    assert np.array_equal(keep.cpu().numpy(), ref)


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 4, 4), (100, 0, 100), (100, 100, 0),
                                                (100, 3, 40), (513, 4, 128), (5000, 4, 100)])
def test_select_shapes(cuda_device, budget, sink, recent):
    check_select(budget, [0, 1, 15, 16, 17, 99, 100, 101, 600, 2047, 513, 514], 3, budget, sink, recent)


@pytest.mark.parametrize("n,budget", [(40001, 10000), (70000, 16384), (5000, 4999), (33000, 1)])
def test_select_long(cuda_device, n, budget):
    check_select(31, [n], 2, budget, min(4, budget // 2), budget // 16)


def test_select_many_tokens_past_shared_memory(cuda_device):
    """A row longer than a cluster keeps in shared memory (8 x 16384 tokens)."""
    check_select(32, [150000, 20], 1, 30001, 4, 1000)


@pytest.mark.parametrize("kind", ["equal", "zero", "negative", "nan", "inf", "denormal", "close"])
def test_select_values(cuda_device, kind):
    def make(w, rng):
        if kind == "equal":
            w[:] = 0.25
        elif kind == "zero":
            w[:] = np.where(rng.rand(*w.shape) < 0.5, 0.0, -0.0)
        elif kind == "negative":
            w[:] = rng.randn(*w.shape)
        elif kind == "nan":
            w[rng.rand(*w.shape) < 0.2] = np.nan
        elif kind == "inf":
            w[rng.rand(*w.shape) < 0.2] = np.inf
            w[rng.rand(*w.shape) < 0.2] = -np.inf
        elif kind == "denormal":
            w[:] = rng.randint(0, 50, w.shape) * np.float32(1e-45)
        else:
            w[:] = 1 + rng.randint(0, 9, w.shape) * np.float32(2.0 ** -23)
    check_select(33, [700, 30, 5000], 2, 300, 4, 64, make)


def test_select_bad_metadata(cuda_device):
    w = torch.rand(8, 2, 16, device="cuda")
    keep = torch.full((2, 2, 10), 77, dtype=torch.int32, device="cuda")
    kl = torch.full((2,), 77, dtype=torch.int32, device="cuda")
    tables = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    ops.get_last_device_error()
    ops.select_tokens(keep, kl, w, tables, torch.tensor([33, 5], dtype=torch.int32).cuda(), 1, 1)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN
    assert kl.tolist() == [0, 5] and bool((keep[0] == -1).all()) and keep[1, 0].tolist() == [0, 1, 2, 3, 4] + [-1] * 5
    tables[0, 1] = 8
    ops.select_tokens(keep, kl, w, tables, torch.tensor([32, 5], dtype=torch.int32).cuda(), 1, 1)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_BLOCK
    assert keep[0, 0, :9].tolist() == sorted(keep[0, 0, :9].tolist()) and int(keep[0, 0, 8]) < 16  # none of the bad block


# ----------------------------------------------------------------- compaction
def check_compact(seed, lens, keep_lens, start, Hkv, D, fp8=False, shared_list=False, with_weights=True, dense=False):
    rng = np.random.RandomState(seed)
    c = U.paged(seed, lens, Hkv, D, fp8)
    heads = 1 if shared_list else Hkv
    mk = max(max(keep_lens), 1) + 2
    keep = np.full((len(lens), heads, mk), -1, np.int32)
    for b, n in enumerate(keep_lens):
        for h in range(heads):
            avail = np.arange(start[b], lens[b])
            if dense:  # the first half stays where it is
                pick = np.concatenate([avail[:n // 2], np.sort(rng.permutation(avail[n // 2:])[:n - n // 2])])
            else:
                pick = np.sort(rng.permutation(avail)[:n])
            keep[b, h, :n] = pick
    w = torch.rand(c.k.shape[:3]) if with_weights else None
    kd, vd, wd = dev(c.k).clone(), dev(c.v).clone(), dev(w).clone() if with_weights else None
    zero = all(s == 0 for s in start)
    ops.compact_kv(kd, vd, dev(c.tables), torch.from_numpy(keep).cuda(), torch.tensor(keep_lens, dtype=torch.int32).cuda(),
                   wd, None if zero else torch.tensor(start, dtype=torch.int32).cuda())
    assert ops.get_last_device_error() == 0
    raw = (lambda x: x.view(torch.uint8)) if fp8 else (lambda x: x)
    for got, x in ((kd, c.k), (vd, c.v)):
        assert U.same_bits(got, U.compact_plain(raw(x), c.tables, keep, keep_lens, start).view(x.dtype))
    if with_weights:
        assert U.same_bits(wd, U.compact_plain(w, c.tables, keep, keep_lens, start))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared_list", [False, True])
@pytest.mark.parametrize("with_weights", [False, True])
def test_compact_shapes(cuda_device, D, fp8, shared_list, with_weights):
    lens = [1, 16, 17, 100, 400, 33, 257, 40]
    check_compact(D, lens, [1, 7, 16, 1, 200, 0, 256, 40], [0] * 8, 2, D, fp8, shared_list, with_weights)


@pytest.mark.parametrize("fp8", [False, True])
def test_compact_drafts(cuda_device, fp8):
    """Accepted paths moved behind prefixes of any length."""
    start = [0, 5, 16, 100, 31]
    check_compact(41, [s + 20 for s in start], [3, 8, 0, 20, 1], start, 3, 128, fp8, shared_list=True, with_weights=False)


@pytest.mark.parametrize("n,m", [(6000, 3001), (6000, 5999), (9000, 20)])
def test_compact_long(cuda_device, n, m):
    """Rows that take several groups of a cluster, moved by a little and by a lot."""
    check_compact(42, [n], [m], [0], 1, 64)
    check_compact(43, [n], [m], [0], 1, 128, fp8=True, dense=True)


def test_compact_many(cuda_device):
    rng = np.random.RandomState(44)
    lens = rng.randint(1, 120, 90)
    check_compact(44, lens.tolist(), [int(rng.randint(0, n + 1)) for n in lens], [0] * 90, 4, 64)


def test_compact_bad_metadata(cuda_device):
    c = U.paged(45, [40, 40, 40], 2, 64)
    kd, vd = dev(c.k).clone(), dev(c.v).clone()
    keep = torch.tensor([[[3, 2, 9]], [[1, 5, 9]], [[0, 4, 700]]], dtype=torch.int32).cuda()
    kl = torch.tensor([3, 99, 3], dtype=torch.int32).cuda()
    ops.get_last_device_error()
    ops.compact_kv(kd, vd, dev(c.tables), keep, kl)
    assert ops.get_last_device_error() == ops.DEVERR_BAD_LEN | ops.DEVERR_BAD_PAIR
    good = [[[3, 1, 9]], [[0, 1, 2]], [[0, 4, 2]]]  # the bad entries stay where they are
    assert U.same_bits(kd, U.compact_plain(c.k, c.tables, np.array(good), [3, 3, 3], [0] * 3))
    assert U.same_bits(vd, U.compact_plain(c.v, c.tables, np.array(good), [3, 3, 3], [0] * 3))
    c.tables[0, 1] = -1
    ops.compact_kv(kd, vd, dev(c.tables), torch.tensor([[[20]], [[0]], [[0]]], dtype=torch.int32).cuda(),
                   torch.tensor([1, 1, 1], dtype=torch.int32).cuda())
    assert ops.get_last_device_error() == ops.DEVERR_BAD_BLOCK


# ------------------------------------------------------------------- together
def test_budgeted_serving(cuda_device):
    """Decode steps that keep weights, a selection, the compaction, decode over
    what is left; then a tree of drafts verified and its accepted path moved
    up: outputs as of a dense cache that holds the kept tokens."""
    B, Hkv, G, D, scale = 3, 2, 4, 64, 0.125
    lens = [50, 90, 20]
    c = U.paged(51, [n + 24 for n in lens], Hkv, D)
    g = torch.Generator().manual_seed(52)
    tables, kd, vd = dev(c.tables), dev(torch.nan_to_num(c.k)).clone(), dev(torch.nan_to_num(c.v)).clone()
    w = torch.full(c.k.shape[:3], math.nan).cuda()
    ws = ops.alloc_weights_workspace(B, Hkv * G, c.tables.shape[1], kd)
    seen = [0] * B
    dense = [[[kd[tables[b].long()[t // 16], h, t % 16].cpu().double() for t in range(lens[b])] for h in range(Hkv)]
             for b in range(B)], [[[vd[tables[b].long()[t // 16], h, t % 16].cpu().double() for t in range(lens[b])]
                                   for h in range(Hkv)] for b in range(B)]
    total = [torch.zeros(Hkv, n, dtype=torch.float64) for n in lens]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    for _ in range(3):
        q = (torch.randn(B, Hkv * G, D, generator=g) * 1.5).bfloat16()
        out = torch.empty_like(q, device="cuda")
        ops.decode_weights(out, w, dev(q), kd, vd, tables, i32(lens), scale, ws, i32(seen))
        seen = list(lens)
        for b in range(B):
            for h in range(Hkv * G):
                k, v = torch.stack(dense[0][b][h // G]), torch.stack(dense[1][b][h // G])
                o, p, av, dot = U.attend64(q[b, h].double(), k, v, scale, torch.ones(lens[b], dtype=torch.bool))
                total[b][h // G] += p
                assert bool(((out[b, h].cpu().double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -11 + U.score_slack(D, dot)) * av).all())
    budget = 32
    keep, kl = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ops.select_tokens(keep, kl, w, tables, i32(lens), 4, 8)
    ops.compact_kv(kd, vd, tables, keep, kl, w)
    kept = keep.cpu()
    lens = kl.tolist()
    assert lens == [32, 32, 20]
    for b in range(B):
        for h in range(Hkv):
            at = [int(t) for t in kept[b, h, :lens[b]]]
            assert at == sorted(set(at)) and at[:4] == [0, 1, 2, 3]
            rest = set(range(total[b].shape[1])) - set(at)
            if rest:  # nothing left out outweighs (by more than the weights' error) what stayed
                mid = [t for t in at if 4 <= t < total[b].shape[1] - 8]
                assert max(float(total[b][h, t]) for t in rest) <= min(float(total[b][h, t]) for t in mid) + 1e-4
            for n in range(2):
                dense[n][b][h] = [dense[n][b][h][t] for t in at]
            got = torch.stack([w[int(c.tables[b, i // 16]), h, i % 16] for i in range(lens[b])]).cpu().double()
            assert bool(((got - total[b][h, at]).abs() <= 1e-4).all())
    # drafts behind the compacted sequences
    T = 6
    newk, newv = torch.randn(B * T, Hkv, D, generator=g).bfloat16(), torch.randn(B * T, Hkv, D, generator=g).bfloat16()
    slots = [int(c.tables[b, (lens[b] + i) // 16]) * 16 + (lens[b] + i) % 16 for b in range(B) for i in range(T)]
    ops.write_kv(dev(newk), dev(newv), torch.tensor(slots).cuda(), kd, vd)
    mask = U.tree_masks(53, [T] * B)
    q = (torch.randn(B * T, Hkv * G, D, generator=g) * 1.5).bfloat16()
    out = torch.empty_like(q, device="cuda")
    tws = ops.alloc_tree_workspace(B, Hkv * G, T, c.tables.shape[1], kd)
    ops.decode_tree(out, dev(q), i32([0, T, 2 * T, 3 * T]), i32(lens), dev(mask), tables, kd, vd, scale, T, tws)
    for b in range(B):
        for h in range(Hkv * G):
            k = torch.stack(dense[0][b][h // G] + [newk[b * T + i, h // G].double() for i in range(T)])
            v = torch.stack(dense[1][b][h // G] + [newv[b * T + i, h // G].double() for i in range(T)])
            for i in range(T):
                see = torch.tensor([True] * lens[b] + [bool((int(mask[b * T + i]) >> j) & 1) for j in range(T)])
                o, _, av, dot = U.attend64(q[b * T + i, h].double(), k, v, scale, see)
                assert bool(((out[b * T + i, h].cpu().double() - o).abs() <=
                             2.0 ** -8 * o.abs() + (2.0 ** -8 + U.score_slack(D, dot)) * av).all())
    path = [0, 2, 5]
    ops.compact_kv(kd, vd, tables, i32([[[n + i for i in path]] for n in lens]), i32([3] * B), w, i32(lens))
    for b in range(B):
        for i, node in enumerate(path):
            t = lens[b] + i
            for h in range(Hkv):
                assert U.same_bits(kd[int(c.tables[b, t // 16]), h, t % 16], newk[b * T + node, h])
                assert U.same_bits(vd[int(c.tables[b, t // 16]), h, t % 16], newv[b * T + node, h])
    assert ops.get_last_device_error() == 0


def test_compaction_beside_a_fork(cuda_device):
    """A sequence that shares its blocks with another gets copies before its
    tokens are moved; the other one's cache keeps its bits."""
    from paged_kv_cache_408_b200.runtime import BlockAllocator, Scheduler, SchedulerConfig, check_invariants
    Hkv, D = 2, 64
    sc = Scheduler(BlockAllocator(24), SchedulerConfig(watermark=0.0))
    a = sc.restore(0, 90, 8)
    b = sc.fork(a, 1, 8)
    g = torch.Generator().manual_seed(91)
    k = torch.randn(24, Hkv, 16, D, generator=g).bfloat16()
    kd, vd = dev(k).clone(), dev(k).clone()
    sc.kv.make_private(b, 4)
    pairs = torch.from_numpy(sc.kv.take_copies()).cuda()
    ops.copy_blocks(kd, vd, pairs)
    keep = torch.tensor([[[0, 1, 2, 3] + list(range(50, 90))]], dtype=torch.int32)
    table = torch.tensor([b.block_table], dtype=torch.int32)
    before = kd.cpu().clone()
    ops.compact_kv(kd, vd, dev(table), dev(keep), torch.tensor([44], dtype=torch.int32).cuda())
    sc.kv.truncate(b, 44)
    assert ops.get_last_device_error() == 0 and len(b.block_table) == 3
    want = U.compact_plain(before, table, keep.numpy(), [44], [0])
    assert U.same_bits(kd, want) and U.same_bits(vd, want)
    for x in a.block_table:
        assert U.same_bits(kd[x], k[x])
    check_invariants(sc)


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_past_32_bit_offsets(cuda_device, fp8):
    """A pool whose elements (and, with E4M3, bytes) pass 2^31: the same bits
    from its last blocks as from a small pool."""
    Hkv, G, D, n, T = 8, 4, 128, 300, 5
    c, q, cu, prefix, mask, scale = make_tree(95, [n], [T], Hkv, G, D, fp8)
    small = c.k.shape[0]
    big = (1 << 31) // (Hkv * 16 * D) + 64 + small
    raw = lambda x: x.view(torch.uint8) if fp8 else x
    pools = []
    for x in (c.k, c.v):
        y = torch.zeros(big, Hkv, 16, D, dtype=raw(x).dtype, device="cuda")
        y[big - small:] = raw(x).cuda()
        pools.append(y.view(x.dtype))
    high = torch.where(c.tables >= 0, c.tables + (big - small), c.tables)
    h = U.Paged(pools[0], pools[1], high, c.k_scale, c.v_scale)
    assert U.same_bits(run_tree(h, q, cu, prefix, mask, scale), run_tree(c, q, cu, prefix, mask, scale))
    w = torch.rand(c.k.shape[:3])
    wh = torch.zeros(big, Hkv, 16)
    wh[big - small:] = w
    a, b = run_weights(c, q[:1], [n], scale, w, [n - 1]), run_weights(h, q[:1], [n], scale, wh, [n - 1])
    assert U.same_bits(a[0], b[0]) and U.same_bits(a[1], b[1][big - small:])
    keep = torch.zeros(2, 1, Hkv, 100, dtype=torch.int32, device="cuda")
    kl = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    ops.select_tokens(keep[0], kl[0], dev(a[1]), dev(c.tables), lens, 4, 20)
    ops.select_tokens(keep[1], kl[1], dev(b[1]), dev(high), lens, 4, 20)
    assert torch.equal(keep[0], keep[1])
    kk, vv = dev(c.k).clone(), dev(c.v).clone()
    ops.compact_kv(kk, vv, dev(c.tables), keep[0], kl[0])
    ops.compact_kv(pools[0], pools[1], dev(high), keep[1], kl[1])
    assert U.same_bits(pools[0][big - small:], kk) and U.same_bits(pools[1][big - small:], vv)
    assert ops.get_last_device_error() == 0


# ------------------------------------------------- streams, graphs, workspaces
def test_calls_in_a_graph_on_another_stream(cuda_device):
    """All four calls captured into one graph on a side stream and replayed
    with new inputs in the same buffers."""
    lens, sizes, Hkv, G, D = [70, 33], [5, 9], 2, 4, 64
    c, q, cu, prefix, mask, scale = make_tree(61, lens, sizes, Hkv, G, D)
    qd, kd, vd, tables = dev(q), dev(c.k), dev(c.v), dev(c.tables)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    cud, pre, ld, md = i32(cu), i32(prefix), i32(lens), dev(mask)
    q1 = (torch.randn(2, Hkv * G, D) * 1.5).bfloat16()
    q1d, w = dev(q1), torch.rand(c.k.shape[:3]).cuda()
    w0 = w.clone()
    out, out1 = torch.zeros_like(qd), torch.zeros_like(q1d)
    keep, kl = torch.zeros(2, Hkv, 40, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    tws, wws = ops.alloc_tree_workspace(2, Hkv * G, 9, tables.shape[1], kd), ops.alloc_weights_workspace(2, Hkv * G, tables.shape[1], kd)
    kk, vv = kd.clone(), vd.clone()
    st = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()

    def calls():
        ops.decode_tree(out, qd, cud, pre, md, tables, kd, vd, scale, 9, tws)
        ops.decode_weights(out1, w, q1d, kd, vd, tables, ld, scale, wws, ld)
        ops.select_tokens(keep, kl, w, tables, ld, 2, 8)
        ops.compact_kv(kk, vv, tables, keep, kl)

    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        calls()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr, stream=st):
        calls()
    for rep in range(2):
        g = torch.Generator().manual_seed(62 + rep)
        q = (torch.randn(q.shape, generator=g) * 1.5).bfloat16()
        q1 = (torch.randn(q1.shape, generator=g) * 1.5).bfloat16()
        qd.copy_(q), q1d.copy_(q1), w.copy_(w0), kk.copy_(kd), vv.copy_(vd)
        gr.replay()
        torch.cuda.synchronize()
        ref, tol = U.tree64(c, q, cu, prefix, mask, scale, 2.0 ** -8)
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
        ref, tol, wr, wtol = U.weights64(c, q1, lens, scale, w0.cpu(), lens)
        assert bool(((out1.cpu().double() - ref).abs() <= tol).all())
        on = wtol > 0
        assert bool(((w.cpu().double() - wr).abs()[on] <= wtol[on]).all())
        rk, rl = U.select_plain(w.cpu().numpy(), c.tables.numpy(), lens, 40, 2, 8)
        assert np.array_equal(keep.cpu().numpy(), rk) and np.array_equal(kl.cpu().numpy(), rl)
        assert U.same_bits(kk, U.compact_plain(c.k, c.tables, rk, rl, [0, 0]))
        assert U.same_bits(vv, U.compact_plain(c.v, c.tables, rk, rl, [0, 0]))
    assert ops.get_last_device_error() == 0


def test_two_streams_at_once(cuda_device):
    """Calls on two streams, each with its own workspace, do not disturb one another."""
    cases = [make_tree(71 + i, [900, 40], [16, 5], 2, 4, 64) for i in range(2)]
    refs = [U.tree64(c, q, cu, p, m, s, 2.0 ** -8) for c, q, cu, p, m, s in cases]
    work = []
    for c, q, cu, p, m, s in cases:
        kd = dev(c.k)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
        qd = dev(q)
        work.append((torch.zeros_like(qd), qd, i32(cu), i32(p), dev(m), dev(c.tables), kd, dev(c.v), s, 16,
                     ops.alloc_tree_workspace(2, 8, 16, c.tables.shape[1], kd)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for st, a in zip(streams, work):
            ops.decode_tree(*a, stream=st)
    torch.cuda.synchronize()
    for a, (ref, tol) in zip(work, refs):
        assert bool(((a[0].cpu().double() - ref).abs() <= tol).all())
    assert ops.get_last_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_repeatable_under_load(cuda_device, fp8, D):
    """Every SM busy with many tiles: the same bits from every call, and the
    right ones (a tile overwritten too early shows here, not on a few tiles)."""
    B, n, T, Hkv, G = 40, 1000, 36, 4, 8
    c = U.paged(83, [n + T] * B, Hkv, D, fp8)
    g = torch.Generator().manual_seed(84)
    q = (torch.randn(B * T, Hkv * G, D, generator=g) * 1.5).bfloat16()
    mask = U.tree_masks(85, [T] * B)
    cu, prefix = [i * T for i in range(B + 1)], [n] * B
    first = run_tree(c, q, cu, prefix, mask, 1 / math.sqrt(D))
    for _ in range(4):
        assert U.same_bits(run_tree(c, q, cu, prefix, mask, 1 / math.sqrt(D)), first)
    for b in (0, 17, 39):
        one = U.Paged(c.k, c.v, c.tables[b:b + 1], c.k_scale, c.v_scale)
        rows = slice(b * T, (b + 1) * T)
        ref, tol = U.tree64(one, q[rows], [0, T], [n], mask[rows], 1 / math.sqrt(D), 2.0 ** -11 if fp8 else 2.0 ** -8)
        assert bool(((first[rows].double() - ref).abs() <= tol).all())


def test_bitwise_repeatable(cuda_device):
    """The same call twice gives the same bits (no order of threads or atomics shows)."""
    c, q, cu, prefix, mask, scale = make_tree(81, [2000, 60], [30, 3], 2, 4, 128)
    assert U.same_bits(run_tree(c, q, cu, prefix, mask, scale), run_tree(c, q, cu, prefix, mask, scale))
    c = U.paged(82, [3000, 40], 2, 128)
    q = torch.randn(2, 8, 128).bfloat16()
    w = torch.rand(c.k.shape[:3])
    a, b = (run_weights(c, q, [3000, 40], 0.1, w, [2999, 39]) for _ in range(2))
    assert U.same_bits(a[0], b[0]) and U.same_bits(a[1], b[1])
