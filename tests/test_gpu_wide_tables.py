"""Block tables wider than any sequence of the batch (a scheduler's tables have
one width): tree attention, decode with weights, selection and compaction give
the plain form's results, and write nothing else."""
import math

import numpy as np
import pytest
import torch

import cache_ops_util as U
from paged_kv_cache_408_b200 import ops
from test_gpu_cache_ops import check_select, check_tree, dev, make_tree, run_weights

pytestmark = pytest.mark.gpu
WIDTHS = [300, 512, 8192]  # 4,800 to 131,072 positions


def widen(c, width):
    t = torch.full((c.tables.shape[0], width), -1, dtype=torch.int32)
    t[:, :c.tables.shape[1]] = c.tables
    c.tables = t
    return c


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("fp8", [False, True])
def test_tree(cuda_device, fp8, width):
    c, *rest = make_tree(101, [0, 3, 700, 128, 16], [5, 0, 33, 64, 1], 2, 4, 64, fp8)
    check_tree(widen(c, width), *rest, pad_rows=2)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("fp8,G", [(False, 4), (True, 8)])
def test_weights(cuda_device, fp8, G, width):
    lens, D = [1, 0, 700, 33, 256], 64
    c = widen(U.paged(102, lens, 2, D, fp8), width)
    g = torch.Generator().manual_seed(103)
    q = (torch.randn(len(lens), 2 * G, D, generator=g) * 1.5).bfloat16()
    w = torch.rand(c.k.shape[:3], generator=g) * 3
    seen = [max(n - 1, 0) for n in lens]
    out, wd = run_weights(c, q, lens, 1 / math.sqrt(D), w, seen)
    assert ops.get_last_device_error() == 0
    ref, tol, wr, wtol = U.weights64(c, q, lens, 1 / math.sqrt(D), w, seen)
    assert bool(((out.double() - ref).abs() <= tol).all())
    on = wtol > 0
    assert U.same_bits(wd[~on], w[~on]) and bool(((wd.double() - wr).abs()[on] <= wtol[on]).all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (16, 4, 4), (100, 0, 100), (513, 4, 128), (6000, 4, 100)])
def test_select(cuda_device, budget, sink, recent, width):
    check_select(104 + budget, [0, 1, 16, 17, 101, 600, 4700], 2, budget, sink, recent, width=width)


@pytest.mark.parametrize("width", WIDTHS)
def test_select_equal_weights(cuda_device, width):
    def make(w, rng):
        w[:] = 0.25
    check_select(105, [4700, 30, 700, 2], 3, 300, 4, 64, make, width=width)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("fp8", [False, True])
def test_compact(cuda_device, fp8, width):
    lens, n = [1, 400, 33, 4700], [1, 200, 0, 1200]
    c = widen(U.paged(106, lens, 2, 64, fp8), width)
    rng = np.random.RandomState(107)
    keep = np.full((4, 2, 1200), -1, np.int32)
    for b in range(4):
        for h in range(2):
            keep[b, h, :n[b]] = np.sort(rng.permutation(lens[b])[:n[b]])
    w = torch.rand(c.k.shape[:3])
    kd, vd, wd = dev(c.k).clone(), dev(c.v).clone(), dev(w).clone()
    ops.compact_kv(kd, vd, dev(c.tables), torch.from_numpy(keep).cuda(), torch.tensor(n, dtype=torch.int32).cuda(), wd)
    assert ops.get_last_device_error() == 0
    raw = (lambda x: x.view(torch.uint8)) if fp8 else (lambda x: x)
    for got, x in ((kd, c.k), (vd, c.v)):
        assert U.same_bits(got, U.compact_plain(raw(x), c.tables, keep, n, [0] * 4).view(x.dtype))
    assert U.same_bits(wd, U.compact_plain(w, c.tables, keep, n, [0] * 4))
