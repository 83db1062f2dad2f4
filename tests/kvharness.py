"""The paged cache and its attention in 64 bits on the CPU, written from the formats' and the operators' definitions."""
from __future__ import annotations

import math

import numpy as np
import torch

NAMES = {0: "bf16", 1: "mxfp8", 2: "mxfp4"}
TOP = {1: (448.0, 7), 2: (6.0, 13)}


def grid(kind):
    """The non-negative values of the element type, ascending, in the order of their codes."""
    if kind == 1:
        return np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127])
    return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])


def nearest_codes(y, kind):
    """Codes (without sign) of the nearest grid values to y >= 0; a tie goes to the even code."""
    gv = grid(kind)
    hi = np.searchsorted(gv, y).clip(0, len(gv) - 1)
    lo = (hi - 1).clip(0)
    dh, dl = gv[hi] - y, y - gv[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (hi == 0)
    return np.where(up, hi, lo)


def quantise(x, kind):
    """float64 rows [..., dim] -> (codes with sign, one per element; scale codes)."""
    top, cap = TOP[kind]
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(b).max(-1)
    bad = ~np.isfinite(a)
    e = np.full(a.shape, -100)
    for i in np.ndindex(a.shape):
        if not bad[i] and a[i] > 0:
            v = int(math.floor(math.log2(a[i] / top))) - 2
            while a[i] > top * 2.0 ** v:
                v += 1
            e[i] = min(max(v, -100), cap)
    y = np.where(bad[..., None], 0.0, b) * 2.0 ** -e[..., None].astype(float)
    code = nearest_codes(np.minimum(np.abs(y), top), kind)
    code = np.where(bad[..., None], 0, code + np.where(np.signbit(y), 128 if kind == 1 else 8, 0))
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def packed(code, kind):
    return code if kind == 1 else (code[..., 0::2] | (code[..., 1::2] << 4))


def stands_for(code, scale, kind):
    """Packed codes and scale codes -> float64 values."""
    if kind == 2:
        code = np.stack((code & 15, code >> 4), -1).reshape(*code.shape[:-1], -1)
    sign = 128 if kind == 1 else 8
    gv = np.append(grid(kind), np.nan) if kind == 1 else grid(kind)
    v = gv[code % sign] * np.where(code >= sign, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(float) - 127))
    return v * np.repeat(s, 32, -1)


class Cache:
    """A paged cache on the GPU, filled with random rows, and its values in 64 bits."""

    def __init__(self, F, kind, heads, dim, page, n_pages, seed, fill=None):
        g = np.random.default_rng(seed)
        self.kind, self.heads, self.dim, self.page, self.n_pages = kind, heads, dim, page, n_pages
        shape = (n_pages, heads, page, dim)
        self.t, self.value = [], []
        scales = []
        for i in range(2):
            if kind == 0:
                x = torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)
                if fill is not None:
                    x[:] = fill
                self.t.append(x.cuda())
                scales.append(None)
                self.value.append(x.double().numpy())
            else:
                code = g.integers(0, 256, (*shape[:3], dim if kind == 1 else dim // 2)).astype(np.uint8)
                if kind == 1:
                    code[(code & 127) == 127] ^= 1  # no NaN codes
                scale = g.integers(118 if kind == 1 else 124, 121 if kind == 1 else 127, (*shape[:3], dim // 32)).astype(np.uint8)
                if kind == 1:  # keep values of order 1
                    code = np.where((code & 127) > 0x48, code & 0xC7, code).astype(np.uint8)
                    scale = scale + 8
                if fill is not None:
                    scale[:] = 255
                self.t.append(torch.from_numpy(code).cuda())
                scales.append(torch.from_numpy(scale).cuda())
                self.value.append(stands_for(code, scale, kind))
        self.scales = scales
        self.c = F.make_kv_cache(kind, heads, dim, page, n_pages, *self.t, *scales)

    def poison(self, which, page, head, off):
        """Makes a cached row (of k: 0, v: 1) NaN."""
        if self.kind == 0:
            self.t[which][page, head, off] = float("nan")
        else:
            self.scales[which][page, head, off] = 255
        self.value[which][page, head, off] = np.nan

    def rows(self, which, pages, head, length):
        return self.value[which][pages, head].reshape(-1, self.dim)[:length]


def attention(cache, q, q_start, kv_len, table, scale, causal=True, window=0):
    """float64 outputs and log sums.  q: float64 [n][heads][dim].  Rows of no sequence stay NaN."""
    n, heads, dim = q.shape
    out, lse = np.full(q.shape, np.nan), np.full((n, heads), np.nan)
    group = heads // cache.heads
    for s in range(len(kv_len)):
        new, length = q_start[s + 1] - q_start[s], kv_len[s]
        pages = table[s, : -(-length // cache.page)]
        for h in range(heads):
            k, v = (cache.rows(i, pages, h // group, length) for i in (0, 1))
            for i in range(new):
                t, p = q_start[s] + i, length - new + i
                hi = min(length, p + 1) if causal else length
                lo = max(0, p - window + 1) if window else 0
                if hi <= lo:
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                z = scale * (k[lo:hi] @ q[t, h])
                top = z.max()
                e = np.exp(z - top)
                lse[t, h] = top + np.log(e.sum())
                out[t, h] = (e / e.sum()) @ v[lo:hi]
    return out, lse
