"""Tree attention, decode with weights, selection and compaction refuse bad
arguments on the host, before any device work (no compute call is made
here)."""
import ctypes as C

import pytest
import torch

from paged_kv_cache_408_b200 import ops

FAKE = C.c_void_p(0x10000)  # never dereferenced: every call below fails validation or has nothing to do
ODD = C.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def desc(nb=64, hkv=8, bs=16, d=128, dt=0):
    return ops.CacheDesc(nb, hkv, bs, d, dt)


def tree(d=None, B=4, maxb=8, Hq=32, max_q=16, total=40, scale=0.1, scales=None, ws=FAKE, ws_bytes=1 << 40, ptr=FAKE,
         mask=FAKE, null=False):
    d = None if null else d or desc()
    return ops.lib().pa_decode_tree(ptr, ptr, ptr, ptr, mask, ptr, B, maxb, Hq, max_q, total, ptr, ptr, scale, scales,
                                    scales, ws, ws_bytes, C.byref(d) if d else None, None)


def test_tree_refusals():
    assert tree(null=True) == INVALID
    assert tree(desc(bs=8)) == INVALID
    assert tree(desc(d=96)) == UNSUPPORTED
    assert tree(desc(hkv=2)) == UNSUPPORTED              # group of 16
    assert tree(Hq=30) == INVALID
    assert tree(B=5000) == INVALID and tree(B=-1) == INVALID
    assert tree(maxb=0) == INVALID and tree(maxb=(1 << 24) + 1) == INVALID
    assert tree(max_q=65) == INVALID and tree(max_q=-1) == INVALID
    assert tree(total=65) == INVALID                     # more rows than 4 x 16
    assert tree(total=-1) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert tree(scale=s) == INVALID
    assert tree(desc(dt=1)) == INVALID                   # fp8 needs its scales
    assert tree(ptr=None) == INVALID and tree(mask=None) == INVALID and tree(ptr=ODD) == INVALID
    assert tree(desc(nb=(1 << 31) // 16 // 8 + 1)) == UNSUPPORTED  # token rows past 32 bits
    assert tree(B=2048, maxb=1 << 20) == UNSUPPORTED     # a line of work past 32 bits
    assert tree(total=0) == 0                            # nothing to do
    assert tree(B=0, total=0) == 0


def tree_ws(B=4, Hq=32, max_q=16, maxb=8, d=None):
    out = C.c_size_t(0)
    return ops.lib().pa_decode_tree_workspace_size(B, Hq, max_q, maxb, C.byref(d or desc()), C.byref(out)), out.value


def weights_ws(B=4, Hq=32, maxb=8, d=None):
    out = C.c_size_t(0)
    return ops.lib().pa_decode_weights_workspace_size(B, Hq, maxb, C.byref(d or desc()), C.byref(out)), out.value


def test_workspace_sizes():
    assert tree_ws()[0] == 0
    assert tree_ws(max_q=65)[0] == INVALID and tree_ws(Hq=30)[0] == INVALID and tree_ws(d=desc(d=96))[0] == UNSUPPORTED
    rc, n = weights_ws()
    assert rc == 0 and n > 0
    assert weights_ws(maxb=0)[0] == INVALID and weights_ws(d=desc(hkv=2))[0] == UNSUPPORTED
    assert weights_ws(B=2048, maxb=1 << 20)[0] == 0      # sized without overflow


def weights(d=None, B=4, maxb=8, Hq=32, scales=None, ws=FAKE, ws_bytes=1 << 60, ptr=FAKE, w=FAKE, null=False):
    d = None if null else d or desc()
    return ops.lib().pa_decode_weights(ptr, w, ptr, ptr, ptr, ptr, ptr, None, B, maxb, Hq, 0.1, scales, scales, ws,
                                       ws_bytes, C.byref(d) if d else None, None)


def test_weights_refusals():
    assert weights(null=True) == INVALID
    assert weights(desc(d=96)) == UNSUPPORTED
    assert weights(desc(hkv=2)) == UNSUPPORTED and weights(desc(hkv=256), Hq=256) == UNSUPPORTED
    assert weights(Hq=30) == INVALID and weights(B=5000) == INVALID and weights(maxb=0) == INVALID
    assert weights(desc(dt=1)) == INVALID
    assert weights(ptr=None) == INVALID and weights(w=None) == INVALID and weights(w=ODD) == INVALID
    assert weights(ws=None) == WORKSPACE and weights(ws_bytes=16) == WORKSPACE
    assert weights(ws=C.c_void_p(0x10010)) == WORKSPACE  # not 256-byte aligned
    assert weights(B=0) == 0


def select(d=None, B=4, maxb=8, budget=100, sink=4, recent=16, ptr=FAKE, w=FAKE):
    return ops.lib().pa_select_tokens(ptr, ptr, w, ptr, ptr, B, maxb, budget, sink, recent, C.byref(d or desc()), None)


def test_select_refusals():
    assert select(desc(nb=0)) == INVALID
    assert select(B=-1) == INVALID and select(B=5000) == INVALID and select(maxb=0) == INVALID
    assert select(budget=0) == INVALID and select(budget=19) == INVALID  # less than sink + recent
    assert select(budget=(1 << 28) + 1) == INVALID
    assert select(sink=-1) == INVALID and select(recent=-1) == INVALID
    assert select(sink=(1 << 31) - 1, recent=(1 << 31) - 1) == INVALID
    assert select(desc(hkv=129)) == UNSUPPORTED
    assert select(ptr=None) == INVALID and select(w=ODD) == INVALID
    assert select(B=0) == 0


def compact(d=None, B=4, maxb=8, heads=8, mk=10, ptr=FAKE, cache=FAKE):
    return ops.lib().pa_compact_kv(cache, cache, None, ptr, ptr, ptr, None, B, maxb, heads, mk, C.byref(d or desc()), None)


def test_compact_refusals():
    assert compact(desc(d=96)) == UNSUPPORTED and compact(desc(hkv=129), heads=129) == UNSUPPORTED
    assert compact(B=-1) == INVALID and compact(maxb=0) == INVALID and compact(mk=-1) == INVALID
    assert compact(heads=2) == INVALID                   # neither one list nor one a head
    assert compact(mk=(1 << 28) + 1) == INVALID
    assert compact(ptr=None) == INVALID and compact(cache=ODD) == INVALID
    assert compact(B=0) == 0 and compact(mk=0) == 0


def test_binding_refuses_host_tensors():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.decode_tree(q, q, i, i, i, i, k, k, 1.0, 1, i)
    with pytest.raises(ValueError):
        ops.decode_weights(q, i, q, k, k, i, i, 1.0, i)
    with pytest.raises(ValueError):
        ops.select_tokens(i, i, torch.zeros(4, 2, 16), i, i, 0, 0)
    with pytest.raises(ValueError):
        ops.compact_kv(k, k, i, i, i)
