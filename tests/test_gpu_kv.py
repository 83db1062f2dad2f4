"""Paged key/value cache and its attention on the GPU against the 64-bit definitions.

Tolerances.  Writing and reading are exact.  Attention, with u = 2^-8 (half a unit in the last of BF16's 8 significant bits):
 - probabilities are rounded to BF16 once: each term of out moves by at most u |p v|;
 - the output is rounded to BF16 once: u |out|;
 - scores and sums are FP32: a score is a sum of dim products, off by at most (dim + 4) 2^-24 sum|q k| scale, which
   moves every p by that factor (twice, through the sum), plus 2^-21 for exp2 and the sums' order.
So |out - ref| <= u |ref| + (u + 2 d + 2^-20) sum_j p_j |v_j| and |lse - ref| <= d + 2^-20 (1 + |ref|), with
d = 1.01 (dim + 4) 2^-24 max_j sum|q k_j| scale.  sum_j p_j |v_j| <= max |v| of the rows that are seen."""
import numpy as np
import pytest
import torch

import kvharness as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from serving_router_top_dedupe_gb300 import ftmoe

    return ftmoe


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def _empty_cache(F, kind, heads, dim, page, n_pages):
    """A cache whose bytes are all 0xA5 / 0x5A, so that rows that must stay as they are can be seen to."""
    per = {0: 2 * dim, 1: dim, 2: dim // 2}[kind]
    k, v = (torch.full((n_pages, heads, page, per), b, dtype=torch.uint8, device="cuda") for b in (0xA5, 0x5A))
    ks, vs = ((torch.full((n_pages, heads, page, dim // 32), b, dtype=torch.uint8, device="cuda") for b in (0xA5, 0x5A))
              if kind else (None, None))
    view = (lambda t: t.view(torch.bfloat16)) if kind == 0 else (lambda t: t)
    return (k, v, ks, vs), F.make_kv_cache(kind, heads, dim, page, n_pages, view(k), view(v), ks, vs)


def _special_rows(rng, n, heads, dim):
    """Rows with what quantisation can go wrong on: ties, zeros, magnitudes from the smallest to the largest."""
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    flat = x.reshape(-1, 32)
    kinds = [lambda b: b * 0, lambda b: b * 2.0 ** -120, lambda b: b * 2.0 ** 100, lambda b: b * 3e4,
             lambda b: np.where(np.arange(32) == 3, 448.0, np.arange(32) * 0.0625),       # E4M3 ties, subnormals
             lambda b: np.where(np.arange(32) == 5, 6.0, (np.arange(32) - 16) * 0.25),    # E2M1 ties of both signs
             lambda b: np.where(np.arange(32) == 9, 449.0, b), lambda b: np.where(np.arange(32) == 9, -6.03125, b),
             lambda b: np.full(32, -3.0e38), lambda b: b * 1e-39, lambda b: np.where(b > 0, -0.0, 1.0)]
    for i, f in enumerate(kinds):
        if i < len(flat):
            flat[(7 * i) % len(flat)] = f(flat[(7 * i) % len(flat)])
    return _bf(x)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 1, 64), (256, 2, 128), (128, 8, 32)])
@pytest.mark.parametrize("n", [1, 37])
def test_write_and_read_match_the_formats(F, kind, dim, heads, page, n):
    rng = np.random.default_rng(dim + heads + n)
    n_pages = 7
    bytes_, c = _empty_cache(F, kind, heads, dim, page, n_pages)
    before = [None if b is None else b.cpu().numpy().copy() for b in bytes_]
    wide = torch.zeros(n, 2 * heads + 3, dim, dtype=torch.bfloat16, device="cuda")  # a projection's rows
    k, v = _special_rows(rng, n, heads, dim), _special_rows(rng, n, heads, dim)
    wide[:, 1:1 + heads] = k.cuda()
    wide[:, 2 + heads:2 + 2 * heads] = v.cuda()
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 1:
        slots[5] = -1
        slots[n - 1] = -(2 ** 31)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    F.ft_kv_write(c, wide[:, 1:1 + heads], wide[:, 2 + heads:2 + 2 * heads], sl, error_word=word)
    ko, vo = (torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    F.ft_kv_read(c, sl, ko, vo, error_word=word)
    torch.cuda.synchronize()
    assert word.item() == 0
    for i, (x, got) in enumerate(((k, ko), (v, vo))):
        x64 = x.double().numpy()
        want, want_scale = before[i], before[2 + i]
        if kind == 0:
            code, ref = x.view(torch.int16).numpy().view(np.uint8).reshape(n, heads, -1), x64
        else:
            code, scale = K.quantise(x64, kind)
            code = K.packed(code, kind)
            ref = K.stands_for(code, scale, kind)
        for t, s in enumerate(slots):
            if s >= 0:
                want[s // page, :, s % page] = code[t]
                if kind:
                    want_scale[s // page, :, s % page] = scale[t]
        ref = np.where((slots >= 0)[:, None, None], ref, 0.0)
        assert np.array_equal(bytes_[i].cpu().numpy(), want)
        if kind:
            assert np.array_equal(bytes_[2 + i].cpu().numpy(), want_scale)
        assert np.array_equal(got.double().cpu().numpy(), ref)


@pytest.mark.parametrize("kind", [1, 2])
def test_a_block_with_a_nan_or_an_infinity_reads_back_as_nan(F, kind):
    heads, dim = 2, 64
    _, c = _empty_cache(F, kind, heads, dim, 16, 2)
    x = torch.ones(3, heads, dim, dtype=torch.bfloat16)
    x[0, 0, 5], x[1, 1, 40], x[2, 0, 0] = float("nan"), float("inf"), float("-inf")
    slots = torch.tensor([3, 17, 20], dtype=torch.int32, device="cuda")
    F.ft_kv_write(c, x.cuda(), x.cuda(), slots)
    ko, vo = (torch.empty(3, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    F.ft_kv_read(c, slots, ko, vo)
    want = torch.ones(3, heads, 2, 32, dtype=torch.bool)
    want[0, 0, 0] = want[1, 1, 1] = want[2, 0, 0] = False
    for t in (ko, vo):
        t = t.cpu().view(3, heads, 2, 32)
        assert torch.equal(torch.isfinite(t), want) and torch.all(t[want] == 1) and torch.all(torch.isnan(t[~want]))


def test_slots_beyond_the_cache_are_skipped_and_reported(F):
    bytes_, c = _empty_cache(F, 1, 1, 128, 16, 2)
    before = [b.clone() for b in bytes_]
    x = torch.ones(2, 1, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([32, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    F.ft_kv_write(c, x, x, slots, error_word=word)
    assert word.item() == F.FT_DEVERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(bytes_, before))
    word.zero_()
    out = torch.ones(2, 1, 128, dtype=torch.bfloat16, device="cuda")
    F.ft_kv_read(c, slots, out, out.clone(), error_word=word)
    assert word.item() == F.FT_DEVERR_BAD_INDEX and out.abs().max().item() == 0


class Batch:
    """A batch of sequences over a cache, with its reference."""

    def __init__(self, F, kind, heads, kv_heads, dim, page, new, lens, seed=1, causal=True, window=0, scale=None,
                 stale_nan=True, max_new=None, extra_rows=0, wide=False):
        rng = np.random.default_rng(seed)
        pages = [-(-n // page) for n in lens]
        self.cache = K.Cache(F, kind, kv_heads, dim, page, sum(pages) + 2, seed)
        order = rng.permutation(sum(pages)) + 1
        stride = max(pages + [1]) + 1
        table = np.full((len(lens), stride), 2 ** 31 - 1, dtype=np.int32)  # entries beyond a length name no page
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = order[at:at + n]
            at += n
            if stale_nan and n and lens[i] % page:  # what lies behind a length
                for off in range(lens[i] % page, page):
                    for h in range(kv_heads):
                        self.cache.poison(0, table[i, n - 1], h, off)
                        self.cache.poison(1, table[i, n - 1], h, off)
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(self.q_start[-1]) + extra_rows
        self.table, self.lens = table, np.array(lens, dtype=np.int32)
        q = rng.standard_normal((n, heads, dim)).astype(np.float32)
        self.scale = scale if scale is not None else 1 / np.sqrt(dim)
        qw = torch.zeros(n, heads + (3 if wide else 0), dim, dtype=torch.bfloat16, device="cuda")
        self.q_t = qw[:, :heads]
        self.q_t.copy_(_bf(q))
        self.q = self.q_t.double().cpu().numpy()
        ow = torch.full((n, heads + (5 if wide else 0), dim), 77.0, dtype=torch.bfloat16, device="cuda")
        self.out = ow[:, :heads]
        self.lse = torch.full((n, heads), 77.0, device="cuda")
        self.word = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(F.ft_attn_workspace(heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
        self.dev = [torch.from_numpy(x).cuda() for x in (self.q_start, self.lens, self.table)]
        self.args = F.make_attn_args(heads, max_new or max(list(new) + [1]), self.q_t, *self.dev, self.out, self.ws, scale=self.scale,
                                     window=window, causal=causal, lse=self.lse, error_word=self.word)
        self.F, self.causal, self.window, self.heads, self.dim = F, causal, window, heads, dim

    def run(self, stream=None):
        self.F.ft_attn(self.cache.c, self.args, stream=stream)
        torch.cuda.synchronize()
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, rows=None):
        out, lse = self.run()
        assert self.word.item() == 0
        ref, ref_lse = K.attention(self.cache, self.q, self.q_start, self.lens, self.table, self.scale, self.causal, self.window)
        n = int(self.q_start[-1])
        assert np.all(out[n:] == 77.0) and np.all(lse[n:] == 77.0)
        group = self.heads // self.cache.heads
        for s in range(len(self.lens)):
            length = int(self.lens[s])
            pages = self.table[s, : -(-length // self.cache.page)]
            for t in range(self.q_start[s], self.q_start[s + 1]):
                if rows is not None and not rows(s, t - self.q_start[s]):
                    continue
                for h in range(self.heads):
                    r, rl = ref[t, h], ref_lse[t, h]
                    if rl == -np.inf:
                        assert np.all(out[t, h] == 0) and lse[t, h] == -np.inf, (s, t, h)
                        continue
                    k, v = (self.cache.rows(i, pages, h // group, length) for i in (0, 1))
                    d = 1.01 * (self.dim + 4) * 2.0 ** -24 * abs(self.scale) * np.nanmax(np.abs(k) @ np.abs(self.q[t, h]))
                    tol = 2.0 ** -8 * np.abs(r) + (2.0 ** -8 + 2 * d + 2.0 ** -20) * np.nanmax(np.abs(v))
                    assert np.all(np.abs(out[t, h] - r) <= tol), (s, t, h, np.max(np.abs(out[t, h] - r) / tol))
                    assert abs(lse[t, h] - rl) <= d + 2.0 ** -20 * (1 + abs(rl)), (s, t, h, lse[t, h], rl)
        return out, lse


SHAPES = [(4, 4, 64), (6, 2, 128), (7, 1, 128), (16, 2, 256), (16, 1, 64), (40, 2, 64)]


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
@pytest.mark.parametrize("page", [16, 128])
def test_single_tokens_of_ragged_sequences(F, kind, heads, kv_heads, dim, page):
    Batch(F, kind, heads, kv_heads, dim, page, new=[1] * 9, lens=[1, 2, 15, 16, 17, 63, 64, 65, 333], wide=True).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (7, 1, 128), (8, 4, 256)])
@pytest.mark.parametrize("window", [0, 1, 40])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_batches(F, kind, heads, kv_heads, dim, window, causal):
    """No new tokens, no cached ones, more new tokens than cached ones, odd chunks; rows that belong to no sequence."""
    Batch(F, kind, heads, kv_heads, dim, 32, new=[3, 0, 1, 5, 33, 2, 70], lens=[3, 40, 0, 2, 150, 129, 70], window=window,
          causal=causal, extra_rows=2, seed=window).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (3, 1, 64), (4, 2, 256)])
@pytest.mark.parametrize("new,length", [(129, 129), (200, 777), (64, 1000)])
def test_chunks(F, kind, heads, kv_heads, dim, new, length):
    Batch(F, kind, heads, kv_heads, dim, 64, new=[new], lens=[length]).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("max_new", [1, 1000])
def test_any_max_new_gives_the_same_results(F, kind, max_new):
    Batch(F, kind, 8, 2, 128, 16, new=[1, 40, 7], lens=[500, 41, 300], max_new=max_new).check()


def test_many_sequences_and_repeated_calls(F):
    """1024 sequences, and a second call on the same workspace gives the same bits."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 60, 1024).tolist()
    b = Batch(F, 0, 2, 1, 64, 16, new=[1] * 1024, lens=lens)
    o1, l1 = b.check()
    o2, l2 = b.run()
    assert np.array_equal(o1, o2) and np.array_equal(l1, l2)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("new", [1, 300])
def test_long_cache_is_split_and_joined(F, kind, new):
    b = Batch(F, kind, 4, 1, 128, 16, new=[new], lens=[9001])
    keep = {0, new // 2, new - 1}
    o1, l1 = b.check(rows=lambda s, i: i in keep)
    o2, l2 = b.run()
    assert np.array_equal(o1, o2) and np.array_equal(l1, l2)


def test_large_scores_do_not_overflow(F):
    """Scores that grow along the cache by hundreds: the running maximum moves again and again."""
    b = Batch(F, 0, 4, 1, 128, 16, new=[2], lens=[700], scale=5.0, stale_nan=False)
    ramp = torch.linspace(0.1, 30, b.cache.n_pages * 16).reshape(-1, 1, 16, 1).to(torch.bfloat16)
    order = np.argsort(b.table[0, :44])
    x = b.cache.t[0].cpu()
    x[torch.from_numpy(b.table[0, :44].astype(np.int64))] *= ramp[:44]
    b.cache.t[0].copy_(x)
    b.cache.value[0] = x.double().numpy()
    assert len(order) == 44
    b.check()


def test_a_captured_call_follows_its_inputs(F):
    b = Batch(F, 1, 8, 2, 128, 32, new=[1, 1], lens=[70, 300])
    b.check()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        F.ft_attn(b.cache.c, b.args, stream=torch.cuda.current_stream().cuda_stream)
    b.lens[:] = [33, 290]
    b.dev[1].copy_(torch.from_numpy(b.lens))
    b.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = b.out.clone()
    b.check()
    assert torch.equal(got, b.out)


def test_bad_lengths_and_pages_are_reported(F):
    b = Batch(F, 0, 4, 2, 64, 16, new=[1, 1], lens=[40, 40])
    good, _ = b.run()
    b.dev[2][0, 1] = b.cache.n_pages  # a page that does not exist
    out, _ = b.run()
    assert b.word.item() == F.FT_DEVERR_BAD_INDEX and np.array_equal(out[1], good[1])
    b.word.zero_()
    b.dev[1][1] = 10 ** 6             # a length beyond the table
    b.dev[1][0] = -3
    out, lse = b.run()
    assert b.word.item() == F.FT_DEVERR_BAD_INDEX and np.all(out[0] == 0) and np.all(lse[0] == -np.inf)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(16, 2, 256, 128), (32, 4, 128, 64), (24, 8, 64, 16)])
@pytest.mark.parametrize("length", [1000, 6001])
def test_kernels_for_few_and_for_many_rows_agree(F, kind, heads, kv_heads, dim, page, length):
    """Many items, several to a CTA and several CTAs to an item: both kernels within twice the tolerance of each other
    (each is within one of the definition), and the same bits again."""
    a, b, c = (Batch(F, kind, heads, kv_heads, dim, page, new=[500, 33], lens=[length, 400], max_new=m) for m in (1, 500, 500))
    (o1, l1), (o2, l2), (o3, l3) = a.run(), b.run(), c.run()
    o4, l4 = c.run()
    assert np.array_equal(o2, o3) and np.array_equal(l2, l3) and np.array_equal(o2, o4) and np.array_equal(l2, l4)
    assert a.word.item() == b.word.item() == 0
    k, v = (np.nanmax(np.abs(x)) for x in a.cache.value)
    d = 1.01 * (dim + 4) * 2.0 ** -24 * a.scale * k * np.abs(a.q).sum(-1).max()
    tol = 2.0 ** -8 * np.abs(o1) + (2.0 ** -8 + 2 * d + 2.0 ** -20) * v
    assert np.all(np.abs(o1 - o2) <= 2 * tol)
    assert np.all(np.abs(l1 - l2) <= 2 * (d + 2.0 ** -20 * (1 + np.abs(l1))))


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,new,length,window", [
    (4, 2, 64, 4, 300, 0), (8, 1, 128, 2, 70, 33), (7, 1, 128, 4, 2000, 0), (4, 2, 256, 3, 45, 0),   # few rows
    (4, 1, 64, 140, 400, 50), (8, 1, 128, 60, 200, 0), (16, 2, 256, 40, 130, 0), (8, 1, 128, 300, 1500, 0)])  # chunks
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_values_that_a_row_does_not_see_do_not_matter(F, kind, heads, kv_heads, dim, new, length, window, value):
    """A cached token within the chunk has values (and keys) that are not finite: rows before it, and rows whose window has
    left it behind, are as if it were not there; rows that see it are NaN."""
    b = Batch(F, kind, heads, kv_heads, dim, 16, new=[new, 1], lens=[length, 40], window=window)
    at = length - new + new // 2  # seen by the later half of the new tokens
    page, off = int(b.table[0, at // 16]), at % 16
    for h in range(kv_heads):
        b.cache.poison(0, page, h, off)
        if kind == 0 and value == "inf":
            b.cache.t[1][page, h, off] = float("inf")
        else:
            b.cache.poison(1, page, h, off)
        b.cache.value[1][page, h, off] = 0.0  # for the rows that do not see it
        b.cache.value[0][page, h, off] = 0.0
    def sees(s, i):
        return s == 0 and length - new + i >= at and (not window or at > length - new + i - window)
    out, lse = b.check(rows=lambda s, i: not sees(s, i))
    seeing = [i for i in range(new) if sees(0, i)]
    assert seeing and np.all(np.isnan(out[seeing])) and np.all(np.isnan(lse[seeing]))
