"""Thin ctypes binding of ``libpa.so`` (declared in ``include/pa.h``).

Argument marshalling only: each function checks tensor devices, dtypes and
shapes, turns tensors into raw device pointers and calls the C entry point of
the same name on the current torch stream.  Every step of the computation
runs in the library's CUDA kernels; there is no fallback.  If the library is
missing, ``lib()`` raises immediately.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

BLOCK_SIZE = 16
PA_OK = 0
DTYPE_BF16, DTYPE_FP8_E4M3 = 0, 1

DEVERR_BAD_BLOCK, DEVERR_BAD_SLOT, DEVERR_BAD_LEN, DEVERR_BAD_PAIR, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_LAYOUT = 0x20

EXPORTED = (
    "pa_write_kv", "pa_copy_blocks", "pa_decode_workspace_size", "pa_decode", "pa_prefill_chunk",
    "pa_get_last_device_error", "pa_status_string", "pa_version", "pa_decode_noalloc",
    "pa_decode_cascade_workspace_size", "pa_decode_cascade",
    "pa_decode_tree_workspace_size", "pa_decode_tree", "pa_decode_weights_workspace_size", "pa_decode_weights",
    "pa_select_tokens", "pa_compact_kv", "pa_copy_blocks_weights",
)
MAX_TREE_ROWS = 64


class PAError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


class CacheDesc(C.Structure):
    _fields_ = [("num_blocks", C.c_int64), ("num_kv_heads", C.c_int32), ("block_size", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32)]


_lib = None


def lib():
    """Load libpa.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpa.so not found at {LIB_PATH}: build it with "
                               "`python -m paged_kv_cache_408_b200.build` (no CPU fallback exists)")
        L = C.CDLL(LIB_PATH)
        p, i32, i64, f32, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
        L.pa_write_kv.argtypes = [p, p, p, i64, p, p, p, p, C.POINTER(CacheDesc), p]
        L.pa_copy_blocks.argtypes = [p, p, p, i32, C.POINTER(CacheDesc), p]
        L.pa_copy_blocks_weights.argtypes = [p, p, p, p, i32, C.POINTER(CacheDesc), p]
        L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, C.POINTER(sz)]
        L.pa_decode.argtypes = [p, p, p, p, p, p, i32, i32, i32, f32, p, p, i32, p, sz, C.POINTER(CacheDesc), p]
        L.pa_prefill_chunk.argtypes = [p, p, p, p, p, i32, i32, i32, i32, i32, p, p, f32, p, p,
                                       C.POINTER(CacheDesc), p]
        L.pa_get_last_device_error.argtypes = [C.POINTER(C.c_uint32), p]
        L.pa_decode_noalloc.argtypes = [p, p, p, p, p, p, i32, i32, i32, f32, p, p, i32, C.POINTER(CacheDesc), p]
        L.pa_decode_cascade_workspace_size.argtypes = [i32, i32, i32, i32, C.POINTER(CacheDesc), C.POINTER(sz)]
        L.pa_decode_cascade.argtypes = [p, p, p, p, p, p, i32, i32, i32, f32, p, p, i32, p, sz,
                                        C.POINTER(CacheDesc), p]
        D = C.POINTER(CacheDesc)
        L.pa_decode_tree_workspace_size.argtypes = [i32, i32, i32, i32, D, C.POINTER(sz)]
        L.pa_decode_tree.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, p, p, f32, p, p, p, sz, D, p]
        L.pa_decode_weights_workspace_size.argtypes = [i32, i32, i32, D, C.POINTER(sz)]
        L.pa_decode_weights.argtypes = [p, p, p, p, p, p, p, p, i32, i32, i32, f32, p, p, p, sz, D, p]
        L.pa_select_tokens.argtypes = [p, p, p, p, p, i32, i32, i32, i32, i32, D, p]
        L.pa_compact_kv.argtypes = [p, p, p, p, p, p, p, i32, i32, i32, i32, D, p]
        L.pa_status_string.argtypes = [C.c_int]
        L.pa_status_string.restype = C.c_char_p
        for f in EXPORTED:
            if f != "pa_status_string":
                getattr(L, f).restype = C.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(int(status)).decode()


def _check(fn, rc):
    if rc != PA_OK:
        raise PAError(fn, rc)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _need(t, name, dtype=None, device=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _current(device):
    """The call launches on the current device: its tensors must live there."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")


FP8_TYPES = (torch.uint8, torch.float8_e4m3fn)


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a cache tensor [num_blocks, Hkv, 16, D] (bf16, or uint8 /
    float8_e4m3fn for E4M3)."""
    if k_cache.dim() != 4 or k_cache.shape[2] != BLOCK_SIZE:
        raise ValueError(f"cache must be [num_blocks, Hkv, {BLOCK_SIZE}, D], got {tuple(k_cache.shape)}")
    if k_cache.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif k_cache.dtype in FP8_TYPES:
        dt = DTYPE_FP8_E4M3
    else:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype}")
    nb, hkv, bs, d = k_cache.shape
    return CacheDesc(nb, hkv, bs, d, dt)


def _caches(k_cache, v_cache):
    _need(k_cache, "k_cache", (torch.bfloat16,) + FP8_TYPES)
    _need(v_cache, "v_cache", k_cache.dtype, k_cache.device)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    return cache_desc(k_cache)


def _scales(desc, k_scale, v_scale, device):
    if desc.dtype != DTYPE_FP8_E4M3:
        return None, None
    if k_scale is None or v_scale is None:
        raise ValueError("an fp8 cache needs k_scale and v_scale")
    _need(k_scale, "k_scale", torch.float32, device)
    _need(v_scale, "v_scale", torch.float32, device)
    if k_scale.numel() != desc.num_kv_heads or v_scale.numel() != desc.num_kv_heads:
        raise ValueError("scales must have one entry per kv head")
    return k_scale, v_scale


def write_kv(k, v, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None, stream=None):
    """pa_write_kv: k, v bf16 [T, Hkv, D]; slot_mapping int64 [T]."""
    desc = _caches(k_cache, v_cache)
    dev = k_cache.device
    _need(k, "k", torch.bfloat16, dev)
    _need(v, "v", torch.bfloat16, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    T = slot_mapping.numel()
    if k.shape != (T, desc.num_kv_heads, desc.head_dim) or v.shape != k.shape:
        raise ValueError(f"k/v must be [T={T}, Hkv, D], got {tuple(k.shape)}")
    ks, vs = _scales(desc, k_scale, v_scale, dev)
    _check("pa_write_kv", lib().pa_write_kv(_ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                                            _ptr(ks), _ptr(vs), C.byref(desc), _stream(stream)))


def copy_blocks(k_cache, v_cache, pairs, stream=None, weights=None):
    """pa_copy_blocks: pairs int32 [n, 2] = (src, dst); with the attention
    weights fp32 [num_blocks, Hkv, 16] that decode_weights keeps beside the
    cache, those of the same blocks too (pa_copy_blocks_weights)."""
    desc = _caches(k_cache, v_cache)
    _need(pairs, "pairs", torch.int32, k_cache.device)
    if pairs.numel() % 2:
        raise ValueError("pairs must be [n, 2]")
    if weights is not None:
        w = _token_weights(weights, desc, k_cache.get_device())
        _check("pa_copy_blocks_weights", lib().pa_copy_blocks_weights(
            _ptr(k_cache), _ptr(v_cache), w, _ptr(pairs), pairs.numel() // 2, C.byref(desc), _stream(stream)))
        return
    _check("pa_copy_blocks", lib().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(pairs), pairs.numel() // 2,
                                                  C.byref(desc), _stream(stream)))


def decode_workspace_size(num_seqs, num_q_heads, head_dim, max_blocks_per_seq, partition_tokens=0) -> int:
    out = C.c_size_t(0)
    _check("pa_decode_workspace_size", lib().pa_decode_workspace_size(
        int(num_seqs), int(num_q_heads), int(head_dim), int(max_blocks_per_seq), int(partition_tokens),
        C.byref(out)))
    return int(out.value)


def alloc_workspace(num_seqs, num_q_heads, head_dim, max_blocks_per_seq, partition_tokens=0, device=None):
    """Caller-side helper: a torch buffer large enough for pa_decode (it
    needs no particular contents; zero-filled here only to be deterministic)."""
    n = decode_workspace_size(num_seqs, num_q_heads, head_dim, max_blocks_per_seq, partition_tokens)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale=None, v_scale=None, workspace=None,
           partition_tokens=0, stream=None):
    """pa_decode: q, out bf16 [B, Hq, D]; block_tables int32 [B, max_blocks];
    seq_lens int32 [B]; workspace a uint8 CUDA buffer (see
    decode_workspace_size)."""
    desc = _caches(k_cache, v_cache)
    dev = k_cache.device
    _need(q, "q", torch.bfloat16, dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    B, Hq, D = q.shape
    if out.shape != q.shape or D != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    ks, vs = _scales(desc, k_scale, v_scale, dev)
    ws_bytes = 0
    if workspace is not None:
        _need(workspace, "workspace", None, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("pa_decode", lib().pa_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens), B,
        block_tables.shape[1], Hq, float(scale), _ptr(ks), _ptr(vs), int(partition_tokens), _ptr(workspace),
        ws_bytes, C.byref(desc), _stream(stream)))


def decode_noalloc(out, q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale=None, v_scale=None,
                   partition_tokens=0, stream=None):
    """pa_decode_noalloc: pa_decode without a caller workspace, for callers
    that cannot allocate device memory; the library's fixed 16 MiB scratch is
    used instead (shapes that need more raise PAError with
    PA_ERR_WORKSPACE).  Calls must not overlap on the GPU."""
    desc = _caches(k_cache, v_cache)
    dev = k_cache.device
    _need(q, "q", torch.bfloat16, dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    B, Hq, D = q.shape
    if out.shape != q.shape or D != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    ks, vs = _scales(desc, k_scale, v_scale, dev)
    _check("pa_decode_noalloc", lib().pa_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens), B,
        block_tables.shape[1], Hq, float(scale), _ptr(ks), _ptr(vs), int(partition_tokens), C.byref(desc),
        _stream(stream)))


def cascade_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, prefix_blocks, k_cache) -> int:
    desc = cache_desc(k_cache)
    out = C.c_size_t(0)
    _check("pa_decode_cascade_workspace_size", lib().pa_decode_cascade_workspace_size(
        int(num_seqs), int(num_q_heads), int(max_blocks_per_seq), int(prefix_blocks), C.byref(desc), C.byref(out)))
    return int(out.value)


def alloc_cascade_workspace(num_seqs, num_q_heads, max_blocks_per_seq, prefix_blocks, k_cache):
    """Caller-side helper: a torch buffer large enough for pa_decode_cascade
    (no particular contents needed)."""
    n = cascade_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, prefix_blocks, k_cache)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=k_cache.device)


def decode_cascade(out, q, k_cache, v_cache, block_tables, seq_lens, scale, prefix_blocks, workspace,
                   k_scale=None, v_scale=None, stream=None):
    """pa_decode_cascade: pa_decode for sequences whose first prefix_blocks
    block-table entries are the same physical blocks in every row (the
    shared prefix is attended once per kv head on the tensor cores)."""
    desc = _caches(k_cache, v_cache)
    dev = k_cache.device
    _need(q, "q", torch.bfloat16, dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    _need(workspace, "workspace", None, dev)
    B, Hq, D = q.shape
    if out.shape != q.shape or D != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    ks, vs = _scales(desc, k_scale, v_scale, dev)
    _check("pa_decode_cascade", lib().pa_decode_cascade(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens), B,
        block_tables.shape[1], Hq, float(scale), _ptr(ks), _ptr(vs), int(prefix_blocks), _ptr(workspace),
        workspace.numel() * workspace.element_size(), C.byref(desc), _stream(stream)))


def prefill_chunk(out, q, cu_q_lens, prefix_lens, block_tables, k_cache, v_cache, scale, max_q_len,
                  k_scale=None, v_scale=None, stream=None):
    """pa_prefill_chunk: q, out bf16 [total_q, Hq, D]; cu_q_lens int32 [n+1];
    prefix_lens int32 [n]; block_tables int32 [n, max_blocks]."""
    desc = _caches(k_cache, v_cache)
    dev = k_cache.device
    _need(q, "q", torch.bfloat16, dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(cu_q_lens, "cu_q_lens", torch.int32, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    n = prefix_lens.numel()
    if cu_q_lens.numel() != n + 1 or block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("cu_q_lens must be [n+1], block_tables [n, max_blocks]")
    total, Hq, D = q.shape
    if out.shape != q.shape or D != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    ks, vs = _scales(desc, k_scale, v_scale, dev)
    _check("pa_prefill_chunk", lib().pa_prefill_chunk(
        _ptr(out), _ptr(q), _ptr(cu_q_lens), _ptr(prefix_lens), _ptr(block_tables), n, block_tables.shape[1], Hq,
        int(max_q_len), total, _ptr(k_cache), _ptr(v_cache), float(scale), _ptr(ks), _ptr(vs), C.byref(desc),
        _stream(stream)))


# The calls below are short enough on the GPU (5-20 us) for the binding itself
# to count: arguments are checked with one expression each, and go through the
# full checks of _need, which say what is wrong, only where that fails.
def _arg(t, name, dtype, index):
    """Device pointer of a contiguous tensor of `dtype` on CUDA device `index`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", index))
    return t.data_ptr()


def _buffer(t, name, index):
    """(pointer, bytes) of a workspace."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.is_contiguous()):
        _need(t, name, None, torch.device("cuda", index))
    return t.data_ptr(), t.numel() * t.element_size()


def _device_index(t, name):
    """The tensor's device, which has to be the current one."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _need(t, name)
    _current(t.device)
    return t.get_device()


def _kv(k_cache, v_cache):
    """(descriptor, device index, k pointer, v pointer)."""
    index = _device_index(k_cache, "k_cache")
    desc = cache_desc(k_cache)
    if not k_cache.is_contiguous():
        _need(k_cache, "k_cache")
    v = _arg(v_cache, "v_cache", k_cache.dtype, index)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    return desc, index, k_cache.data_ptr(), v


def _scale_args(desc, k_scale, v_scale, index):
    if desc.dtype != DTYPE_FP8_E4M3:
        return None, None
    k_scale, v_scale = _scales(desc, k_scale, v_scale, torch.device("cuda", index))
    return k_scale.data_ptr(), v_scale.data_ptr()


def _raw_stream(stream, index):
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _token_weights(weights, desc, index):
    w = _arg(weights, "weights", torch.float32, index)
    if weights.shape != (desc.num_blocks, desc.num_kv_heads, BLOCK_SIZE):
        raise ValueError(f"weights must be [num_blocks, Hkv, {BLOCK_SIZE}], got {tuple(weights.shape)}")
    return w


def tree_workspace_size(num_seqs, num_q_heads, max_q_len, max_blocks_per_seq, k_cache) -> int:
    desc = cache_desc(k_cache)
    out = C.c_size_t(0)
    _check("pa_decode_tree_workspace_size", lib().pa_decode_tree_workspace_size(
        int(num_seqs), int(num_q_heads), int(max_q_len), int(max_blocks_per_seq), C.byref(desc), C.byref(out)))
    return int(out.value)


def alloc_tree_workspace(num_seqs, num_q_heads, max_q_len, max_blocks_per_seq, k_cache):
    """Caller-side helper: a torch buffer large enough for pa_decode_tree (no
    particular contents needed)."""
    n = tree_workspace_size(num_seqs, num_q_heads, max_q_len, max_blocks_per_seq, k_cache)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=k_cache.device)


def decode_tree(out, q, cu_q_lens, prefix_lens, mask, block_tables, k_cache, v_cache, scale, max_q_len, workspace,
                k_scale=None, v_scale=None, stream=None):
    """pa_decode_tree: q, out bf16 [total_q, Hq, D]; cu_q_lens int32 [n+1];
    prefix_lens int32 [n]; mask int64 (or uint64) [total_q], bit j = the row
    sees draft j of its sequence; block_tables int32 [n, max_blocks]; at most
    MAX_TREE_ROWS drafts a sequence."""
    desc, dev, kp, vp = _kv(k_cache, v_cache)
    qp, op = _arg(q, "q", torch.bfloat16, dev), _arg(out, "out", torch.bfloat16, dev)
    cp, pp = _arg(cu_q_lens, "cu_q_lens", torch.int32, dev), _arg(prefix_lens, "prefix_lens", torch.int32, dev)
    uint64 = isinstance(mask, torch.Tensor) and mask.dtype is torch.uint64
    mp = _arg(mask, "mask", torch.uint64 if uint64 else torch.int64, dev)
    tp = _arg(block_tables, "block_tables", torch.int32, dev)
    wp, wn = _buffer(workspace, "workspace", dev)
    n = prefix_lens.numel()
    if cu_q_lens.numel() != n + 1 or block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("cu_q_lens must be [n+1], block_tables [n, max_blocks]")
    if q.dim() != 3 or out.shape != q.shape or q.shape[2] != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    total, Hq, _ = q.shape
    if mask.dim() != 1 or mask.shape[0] != total:
        raise ValueError("mask must be [total_q]")
    ks, vs = _scale_args(desc, k_scale, v_scale, dev)
    _check("pa_decode_tree", lib().pa_decode_tree(
        op, qp, cp, pp, mp, tp, n, block_tables.shape[1], Hq, int(max_q_len), total, kp, vp, float(scale), ks, vs, wp, wn,
        C.byref(desc), _raw_stream(stream, dev)))


def weights_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, k_cache) -> int:
    desc = cache_desc(k_cache)
    out = C.c_size_t(0)
    _check("pa_decode_weights_workspace_size", lib().pa_decode_weights_workspace_size(
        int(num_seqs), int(num_q_heads), int(max_blocks_per_seq), C.byref(desc), C.byref(out)))
    return int(out.value)


def alloc_weights_workspace(num_seqs, num_q_heads, max_blocks_per_seq, k_cache):
    """Caller-side helper: a torch buffer large enough for pa_decode_weights
    (no particular contents needed)."""
    n = weights_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, k_cache)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=k_cache.device)


def decode_weights(out, weights, q, k_cache, v_cache, block_tables, seq_lens, scale, workspace, seen_lens=None,
                   k_scale=None, v_scale=None, stream=None):
    """pa_decode_weights: decode that adds every cached token's attention
    weight, summed over its kv head's query heads, to weights fp32
    [num_blocks, Hkv, 16]; seen_lens int32 [B] (positions whose sum is there
    already; None: all of them)."""
    desc, dev, kp, vp = _kv(k_cache, v_cache)
    qp, op = _arg(q, "q", torch.bfloat16, dev), _arg(out, "out", torch.bfloat16, dev)
    tw = _token_weights(weights, desc, dev)
    tp, lp = _arg(block_tables, "block_tables", torch.int32, dev), _arg(seq_lens, "seq_lens", torch.int32, dev)
    wp, wn = _buffer(workspace, "workspace", dev)
    if q.dim() != 3 or out.shape != q.shape or q.shape[2] != desc.head_dim:
        raise ValueError("out/q shape mismatch")
    B, Hq, _ = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    sp = None
    if seen_lens is not None:
        sp = _arg(seen_lens, "seen_lens", torch.int32, dev)
        if seen_lens.shape != (B,):
            raise ValueError("seen_lens must be [B]")
    ks, vs = _scale_args(desc, k_scale, v_scale, dev)
    _check("pa_decode_weights", lib().pa_decode_weights(
        op, tw, qp, kp, vp, tp, lp, sp, B, block_tables.shape[1], Hq, float(scale), ks, vs, wp, wn, C.byref(desc),
        _raw_stream(stream, dev)))


def select_tokens(keep, keep_lens, weights, block_tables, seq_lens, num_sink, num_recent, stream=None):
    """pa_select_tokens: the positions each kv head keeps under a budget
    (keep int32 [B, Hkv, budget], ascending, then -1; keep_lens int32 [B]):
    the first num_sink, the last num_recent, the heaviest of the rest by
    weights fp32 [num_blocks, Hkv, 16]."""
    dev = _device_index(weights, "weights")
    wp = _arg(weights, "weights", torch.float32, dev)
    kp, np_ = _arg(keep, "keep", torch.int32, dev), _arg(keep_lens, "keep_lens", torch.int32, dev)
    tp, lp = _arg(block_tables, "block_tables", torch.int32, dev), _arg(seq_lens, "seq_lens", torch.int32, dev)
    if weights.dim() != 3 or weights.shape[2] != BLOCK_SIZE:
        raise ValueError(f"weights must be [num_blocks, Hkv, {BLOCK_SIZE}], got {tuple(weights.shape)}")
    nb, hkv, bs = weights.shape
    B = seq_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B or keep_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks], seq_lens and keep_lens [B]")
    if keep.dim() != 3 or keep.shape[:2] != (B, hkv):
        raise ValueError("keep must be [B, Hkv, budget]")
    desc = CacheDesc(nb, hkv, bs, 128, DTYPE_BF16)  # the call reads num_blocks and num_kv_heads only
    _check("pa_select_tokens", lib().pa_select_tokens(
        kp, np_, wp, tp, lp, B, block_tables.shape[1], keep.shape[2], int(num_sink), int(num_recent), C.byref(desc),
        _raw_stream(stream, dev)))


def compact_kv(k_cache, v_cache, block_tables, keep, keep_lens, weights=None, start_lens=None, stream=None):
    """pa_compact_kv: K and V (and the weights, if given) of position
    keep[b, head, i] move to position start_lens[b] + i, in place; keep int32
    [B, Hkv or 1, max_keep] ascending, keep_lens int32 [B], start_lens int32
    [B] (None: 0)."""
    desc, dev, kp, vp = _kv(k_cache, v_cache)
    tp = _arg(block_tables, "block_tables", torch.int32, dev)
    lp, np_ = _arg(keep, "keep", torch.int32, dev), _arg(keep_lens, "keep_lens", torch.int32, dev)
    B = keep_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [B, max_blocks]")
    if keep.dim() != 3 or keep.shape[0] != B:
        raise ValueError("keep must be [B, Hkv or 1, max_keep]")
    wp = None if weights is None else _token_weights(weights, desc, dev)
    sp = None
    if start_lens is not None:
        sp = _arg(start_lens, "start_lens", torch.int32, dev)
        if start_lens.shape != (B,):
            raise ValueError("start_lens must be [B]")
    _check("pa_compact_kv", lib().pa_compact_kv(
        kp, vp, wp, tp, lp, np_, sp, B, block_tables.shape[1], keep.shape[1], keep.shape[2], C.byref(desc),
        _raw_stream(stream, dev)))


def get_last_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    flags = C.c_uint32(0)
    rc = lib().pa_get_last_device_error(C.byref(flags), _stream(stream))
    if rc not in (PA_OK, -5):
        raise PAError("pa_get_last_device_error", rc)
    return int(flags.value)
