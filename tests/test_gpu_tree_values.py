"""Tree attention over values and scales at the ends of their ranges, against
the plain form in 64 bits."""
import math

import pytest
import torch

import cache_ops_util as U
from paged_kv_cache_408_b200 import ops
from test_gpu_cache_ops import check_tree, make_tree, run_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("prefix,T,G", [
    (70, 6, 2),      # one key tile: one stream alone holds the rows
    (70, 40, 4),     # one key tile, two row tiles
    (700, 40, 4),    # two row tiles over many key tiles
    (700, 6, 2),     # one row tile: the two streams' accumulators are joined
    (9000, 6, 2),    # pieces of many CTAs, merged
])
def test_infinite_value_in_the_prefix(cuda_device, prefix, T, G, value):
    """An infinite V element of a token that every row sees is that infinity
    in every row's output, in its column alone, whatever the split."""
    c, q, cu, pre, mask, scale = make_tree(91, [prefix], [T], 1, G, 64)
    t = prefix // 2
    c.v[int(c.tables[0, t // 16]), 0, t % 16, 5] = value
    out = run_tree(c, q, cu, pre, mask, scale).double()
    assert ops.get_last_device_error() == 0
    assert bool((out[:, :, 5] == value).all())
    ref, tol = U.tree64(c, q, cu, pre, mask, scale, 2.0 ** -8)
    rest = torch.arange(64) != 5
    assert bool(((out - ref).abs()[:, :, rest] <= tol[:, :, rest]).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [2, 8])
def test_any_finite_head_scale(cuda_device, G, D):
    """K scales that are zero (every visible key weighs the same) or negative,
    V scales likewise, in tiles with and without masked keys."""
    c, q, cu, pre, mask, scale = make_tree(92, [0, 100, 1000, 31], [5, 40, 3, 1], 4, G, D, fp8=True)
    c.k_scale = torch.tensor([0.0, -0.013, 0.011, -0.0])
    c.v_scale = torch.tensor([0.012, 0.014, 0.0, -0.01])
    check_tree(c, q, cu, pre, mask, scale)
