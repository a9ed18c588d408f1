"""Inputs and 64-bit plain forms for the tests of tree attention, decode with
attention weights, token selection and compaction (torch on the host)."""
import math
from dataclasses import dataclass

import numpy as np
import torch

BS = 16


@dataclass
class Paged:
    """A scattered paged cache on the host and its block tables."""
    k: torch.Tensor            # [num_blocks, Hkv, 16, D] bf16 or float8_e4m3fn
    v: torch.Tensor
    tables: torch.Tensor       # int32 [B, max_blocks], -1 past a sequence's last block
    k_scale: torch.Tensor = None
    v_scale: torch.Tensor = None

    @property
    def Hkv(self):
        return self.k.shape[1]

    @property
    def D(self):
        return self.k.shape[3]

    def row64(self, name, b, t, h):
        """Token t's K or V row of kv head h in 64 bits."""
        x = getattr(self, name)[int(self.tables[b, t // BS]), h, t % BS].to(torch.float32).double()
        s = getattr(self, name + "_scale")
        return x if s is None else x * s[h].double()

    def rows64(self, name, b, n):
        """[n, Hkv, D] in 64 bits."""
        t = torch.arange(n)
        blk = self.tables[b].long()[t // BS]
        x = getattr(self, name)
        raw = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        y = raw[blk, :, t % BS].view(x.dtype).to(torch.float32).double()
        s = getattr(self, name + "_scale")
        return y if s is None else y * s.double()[:, None]


def paged(seed, lens, Hkv, D, fp8=False, extra_blocks=3, width=None):
    """A pool with `extra_blocks` unused blocks (NaN in them and behind every
    sequence's last token: nothing may read those)."""
    g = torch.Generator().manual_seed(seed)
    nb = [(n + BS - 1) // BS for n in lens]
    pool = sum(nb) + extra_blocks
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    maxb = width or max(max(nb), 1)
    tables = torch.full((len(lens), maxb), -1, dtype=torch.int32)
    used = torch.zeros(pool, BS, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        tables[b, :nb[b]] = perm[at:at + nb[b]]
        for j in range(nb[b]):
            used[int(perm[at + j]), :min(BS, n - j * BS)] = True
        at += nb[b]
    scale = (5.5 / 448) * (1 + 0.125 * torch.arange(Hkv, dtype=torch.float32)) if fp8 else None
    out = []
    for _ in range(2):
        x = torch.randn(pool, Hkv, BS, D, generator=g)
        x = x / scale[:, None, None] if fp8 else x
        x = torch.where(used[:, None, :, None], x, torch.full_like(x, math.nan))
        out.append(x.to(torch.float8_e4m3fn if fp8 else torch.bfloat16))
    return Paged(out[0], out[1], tables, scale, scale)


def tree_masks(seed, sizes):
    """Random trees: node i hangs below one of the four nodes before it."""
    rng = np.random.RandomState(seed)
    rows = []
    for n in sizes:
        m = []
        for i in range(n):
            m.append((m[rng.randint(max(0, i - 4), i)] if i else 0) | (1 << i))
        rows += m
    return torch.from_numpy(np.array(rows, np.uint64).view(np.int64).copy())


def attend64(q, k, v, scale, see):
    """One query row over n keys: (out [D], p [n], sum p |v| [D], largest sum of |q_d k_d|)."""
    if not bool(see.any()):
        z = torch.zeros(q.shape[0], dtype=torch.float64)
        return z, torch.zeros(k.shape[0], dtype=torch.float64), z, 0.0
    s = (k[see] @ q) * scale
    p = torch.softmax(s, 0)
    full = torch.zeros(k.shape[0], dtype=torch.float64)
    full[see] = p
    return p @ v[see], full, p @ v[see].abs(), float((k[see].abs() @ q.abs()).max()) * scale


def score_slack(D, absdot):
    """Relative error of a softmax weight from 32-bit scores: D products summed
    in fp32 (each addition off by 2^-24 of a partial sum of at most absdot),
    once in the weight and once in its normaliser, plus the hardware base-2
    exponential and its argument's rounding (2^-22 and absdot * 2^-23)."""
    return 2 * (D * 2.0 ** -24 * absdot + 2.0 ** -22 + absdot * 2.0 ** -23)


def tree64(c, q, cu, prefix, mask, scale, p_rounding):
    """(out, tolerance) [total, Hq, D].  Tolerance: the bf16 output (2^-8 of
    the value) and, per key, the weight's rounding to the matrix operand's
    type (p_rounding) and its 32-bit score, each relative to the weight."""
    total, Hq, D = q.shape
    G = Hq // c.Hkv
    out = torch.zeros(total, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(len(cu) - 1):
        T, P = cu[b + 1] - cu[b], prefix[b]
        if T == 0:
            continue
        k, v = c.rows64("k", b, P + T), c.rows64("v", b, P + T)
        for i in range(T):
            bits = int(mask[cu[b] + i]) & ((1 << 64) - 1)
            see = torch.ones(P + T, dtype=torch.bool)
            for j in range(T):
                see[P + j] = bool((bits >> j) & 1)
            for h in range(Hq):
                o, _, av, dot = attend64(q[cu[b] + i, h].double(), k[:, h // G], v[:, h // G], scale, see)
                out[cu[b] + i, h] = o
                tol[cu[b] + i, h] = 2.0 ** -8 * o.abs() + (p_rounding + score_slack(D, dot)) * av
    return out, tol


def weights64(c, q, lens, scale, weights, seen):
    """(out, its tolerance, weights, their tolerance)."""
    B, Hq, D = q.shape
    G = Hq // c.Hkv
    out, tol = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    w, wtol = weights.double().clone(), torch.zeros(weights.shape, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        k, v = c.rows64("k", b, n), c.rows64("v", b, n)
        t = torch.arange(n)
        blk = c.tables[b].long()[t // BS]
        for kh in range(c.Hkv):
            got = torch.where(t < int(seen[b]), w[blk, kh, t % BS], torch.zeros(n, dtype=torch.float64))
            err = torch.zeros(n, dtype=torch.float64)
            for h in range(kh * G, (kh + 1) * G):
                if n == 0:
                    continue
                o, p, av, dot = attend64(q[b, h].double(), k[:, kh], v[:, kh], scale, torch.ones(n, dtype=torch.bool))
                out[b, h] = o
                # the tensor-core decode of an fp8 cache rounds weights to f16 for its product
                tol[b, h] = 2.0 ** -8 * o.abs() + (2.0 ** -11 + score_slack(D, dot)) * av
                got, err = got + p, err + p * score_slack(D, dot)
            w[blk, kh, t % BS] = got
            # G additions in fp32, and weights below 2^-126 of the total may be flushed to zero
            wtol[blk, kh, t % BS] = err + (G + 1) * 2.0 ** -24 * got.abs() + 2.0 ** -120
    return out, tol, w, wtol


def select_plain(weights, tables, lens, budget, sink, recent):
    B, Hkv = len(lens), weights.shape[1]
    keep = np.full((B, Hkv, budget), -1, np.int32)
    got = np.zeros(B, np.int32)
    for b in range(B):
        n = int(lens[b])
        got[b] = min(n, budget)
        t = np.arange(n)
        for h in range(Hkv):
            w = weights[tables[b][t // BS], h, t % BS].astype(np.float64)
            w = np.where(np.isnan(w), np.inf, w)
            isn = np.isnan(weights[tables[b][t // BS], h, t % BS])
            if n <= budget:
                pos = list(t)
            else:
                mid = list(range(sink, n - recent))
                mid.sort(key=lambda i: (-w[i], not isn[i], i))  # NaN above +inf; ties to the lowest
                pos = sorted(list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n)))
            keep[b, h, :len(pos)] = pos
    return keep, got


def compact_plain(x, tables, keep, keep_lens, start):
    """x [num_blocks, Hkv, 16, ...] -> a copy with the kept tokens moved."""
    y = x.clone()
    for b in range(len(keep_lens)):
        for h in range(x.shape[1]):
            for i in range(int(keep_lens[b])):
                s, d = int(keep[b, h if keep.shape[1] > 1 else 0, i]), int(start[b]) + i
                y[int(tables[b, d // BS]), h, d % BS] = x[int(tables[b, s // BS]), h, s % BS]
    return y


def same_bits(a, b):
    """Equal bit patterns (NaN included)."""
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return bool(torch.equal(a.cpu().view(view), b.cpu().view(view)))
