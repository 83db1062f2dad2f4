"""64-bit attention with what bounds its rounding column by column, and caches over given values.

Bound of an output element.  With u = 2^-8 (half a unit in the last of BF16's 8 significant bits), n the tokens that a row
sees and A = sum_j p_j |v_j| of that row and column:
 - every term's probability is rounded to BF16 once (with its value's power of two, which does not round): u A;
 - the output is rounded to BF16 once: u |out|;
 - a score is an FP32 sum of dim products, rounded or cut off after each: (dim + 4) 2^-23 sum |q k| scale at most, which moves
   every p by that factor d, twice through the sum;
 - sums of n terms are rounded or cut off after each: n 2^-23 A; exp2 and the factors between parts: 2^-16 A is ample;
 - numbers below FP32's normal range, 2^-126, may be lost where sums are held relative to 2^-22 of their value: n 2^-104 A'
   with A' = max |v| / 2^7 of the column's 32-column block in the format, which the caller adds where scales go that low.
|lse - ref| <= d + n 2^-23 + 2^-20 (1 + |ref|)."""
from __future__ import annotations

import numpy as np
import torch

import kvharness as K

U = 2.0 ** -8


class Cache(K.Cache):
    """A paged cache on the GPU that holds the given rows ([n_pages][heads][page][dim] float64, quantised as the format says)."""

    def __init__(self, F, kind, k, v):
        self.kind, (self.n_pages, self.heads, self.page, self.dim) = kind, k.shape
        self.t, self.scales, self.value = [], [], []
        for x in (k, v):
            if kind == 0:
                b = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
                self.t.append(b.cuda())
                self.scales.append(None)
                self.value.append(b.double().numpy())
            else:
                code, scale = K.quantise(x, kind)
                code = K.packed(code, kind)
                self.t.append(torch.from_numpy(np.ascontiguousarray(code)).cuda())
                self.scales.append(torch.from_numpy(scale).cuda())
                self.value.append(K.stands_for(code, scale, kind))
        self.c = F.make_kv_cache(kind, self.heads, self.dim, self.page, self.n_pages, *self.t, *self.scales)


def attention(cache, q, q_start, kv_len, table, scale, causal=True, window=0, rows=None):
    """For every row that a sequence names (rows(s, i): only those): out, A and the score bound d, n, all float64 (NaN
    elsewhere).  Unseen tokens are left out, not multiplied by zero."""
    n, heads, dim = q.shape
    out, mass = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, d, seen = (np.full((n, heads), np.nan) for _ in range(3))
    group = heads // cache.heads
    for s in range(len(kv_len)):
        new, length = int(q_start[s + 1] - q_start[s]), int(kv_len[s])
        pages = table[s, : -(-length // cache.page)]
        for kh in range(cache.heads):
            k, v = (cache.rows(i, pages, kh, length) for i in (0, 1))
            for i in range(new):
                if rows is not None and not rows(s, i):
                    continue
                t, p = q_start[s] + i, length - new + i
                hi = min(length, p + 1) if causal else length
                lo = max(0, p - window + 1) if window else 0
                h = slice(kh * group, (kh + 1) * group)
                seen[t, h] = max(hi - lo, 0)
                if hi <= lo:
                    out[t, h], mass[t, h], lse[t, h], d[t, h] = 0.0, 0.0, -np.inf, 0.0
                    continue
                z = scale * (q[t, h] @ k[lo:hi].T)
                top = z.max(-1, keepdims=True)
                e = np.exp(z - top)
                total = e.sum(-1, keepdims=True)
                lse[t, h] = (top + np.log(total))[:, 0]
                out[t, h] = (e / total) @ v[lo:hi]
                mass[t, h] = (e / total) @ np.abs(v[lo:hi])
                d[t, h] = (dim + 4) * 2.0 ** -23 * abs(scale) * (np.abs(q[t, h]) @ np.abs(k[lo:hi]).T).max(-1)
    return out, mass, lse, d, seen


def check(got, got_lse, ref, floor=0.0):
    """Every element of the rows that ref has (attention()'s results) within its bound; floor: added to it, [dim] or a number."""
    out, mass, lse, d, n = ref
    rows = ~np.isnan(n)
    assert rows.any()
    with np.errstate(invalid="ignore"):
        tol = U * np.abs(out) + (U + 2 * d + n * 2.0 ** -23 + 2.0 ** -16)[..., None] * mass + floor
        bad = ~(np.abs(got - out) <= tol)[rows]
        assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:3], got[rows][bad][:3], out[rows][bad][:3], tol[rows][bad][:3])
        none = rows & (n == 0)
        assert np.all(got_lse[none] == -np.inf)
        some = rows & (n > 0)
        ltol = d + n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(lse))
        worst = (np.abs(got_lse - lse) / ltol)[some]
        assert np.all(worst <= 1), np.max(worst)


class Call:
    """ft_attn of a batch over a cache: sequence s has new[s] tokens and lens[s] cached ones, in the pages that table names.
    wide: more entries in every row of the table, naming no page, so that there might be much to read.  copies: whether the
    workspace has room for decoded pages."""

    def __init__(self, F, cache, heads, new, lens, table=None, scale=None, causal=True, window=0, wide=0, q=None, max_new=None, seed=1,
                 copies=True):
        rng = np.random.default_rng(seed)
        if table is None:  # pages in an order of their own
            pages = [-(-n // cache.page) for n in lens]
            order = rng.permutation(sum(pages))
            table = np.full((len(lens), max(pages + [1])), -1, dtype=np.int32)
            for s, n in enumerate(pages):
                at = sum(pages[:s])
                table[s, :n] = order[at:at + n]
        self.F, self.cache, self.causal, self.window, self.table = F, cache, causal, window, table
        self.scale = 1 / np.sqrt(cache.dim) if scale is None else scale
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        n = int(self.q_start[-1])
        q = rng.standard_normal((n, heads, cache.dim)) if q is None else q
        self.q_t = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16).cuda()
        self.q = self.q_t.double().cpu().numpy()
        self.out, self.lse = torch.full_like(self.q_t, 77.0), torch.full((n, heads), 77.0, device="cuda")
        self.word = torch.zeros(1, dtype=torch.int32, device="cuda")
        bytes_ = F.ft_attn_workspace(heads, cache.heads, cache.dim) - (0 if copies else 512 << 20)
        self.ws = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
        full = np.concatenate([table, np.full((len(lens), wide), 2 ** 31 - 1, dtype=np.int32)], 1)
        self.dev = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (self.q_start, self.lens, full)]
        self.args = F.make_attn_args(heads, max_new or max(new), self.q_t, *self.dev, self.out, self.ws, scale=self.scale,
                                     window=window, causal=causal, lse=self.lse, error_word=self.word)

    def run(self, cache=None):
        self.F.ft_attn((cache or self.cache).c, self.args)
        torch.cuda.synchronize()
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def reference(self, rows=None):
        return attention(self.cache, self.q, self.q_start, self.lens, self.table, self.scale, self.causal, self.window, rows)

    def check(self, rows=None, floor=0.0):
        got = self.run()
        assert self.word.item() == 0
        check(*got, self.reference(rows), floor)
        return got
