"""Attention over the paged cache where single rows, blocks or columns are out of the ordinary: pages that do not exist,
values that are no numbers, scales far apart.  Bounds: kvexact.py."""
import numpy as np
import pytest
import torch

import kvexact as X
import kvharness as K
from test_gpu_kv import F  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

WIDE = 40000  # table entries that make a chunk of a hundred rows go to the kernel for many rows


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("new,bad", [(1, [0]), (3, [0]), (1, [0, 1, 2, 3]), (1, [0, 2, 5])])
def test_bad_pages_under_few_rows_count_as_zeros(F, kind, heads, kv_heads, dim, page, new, bad):
    """Whole pages that name nothing, the first ones that a row sees among them: the same bits as with pages of zeros."""
    cache = K.Cache(F, kind, kv_heads, dim, page, 9, 4)
    call = X.Call(F, cache, heads, [new, new], [7 * page + 5, page + 3], table=np.array([range(8), [8, 3] + [-1] * 6], dtype=np.int32))
    for i in bad:
        call.dev[2][0, i] = cache.n_pages + i
    got = call.run()
    assert call.word.item() == F.FT_DEVERR_BAD_INDEX
    assert all(np.all(np.isfinite(x)) for x in got)
    zero = [t.clone() for t in cache.t]
    for t in zero:
        t[bad] = 0
    call.dev[2][0, bad] = torch.tensor(bad, dtype=torch.int32, device="cuda")
    call.word.zero_()
    F.ft_attn(F.make_kv_cache(kind, kv_heads, dim, page, cache.n_pages, *zero, *cache.scales), call.args)
    torch.cuda.synchronize()
    assert call.word.item() == 0
    n = new  # rows of the sequence whose pages were bad; the other's page 3 is one of the zeroed ones where bad has it
    assert np.array_equal(call.out.double().cpu().numpy()[:n], got[0][:n]) and np.array_equal(call.lse.double().cpu().numpy()[:n], got[1][:n])


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("new,length,wide", [(1, 1, 0), (1, 300, 0), (4, 70, 0), (70, 90, WIDE)])
def test_log_sums_do_not_depend_on_values(F, kind, heads, kv_heads, dim, new, length, wide):
    """All values NaN: out is NaN, and lse is that of the keys."""
    cache = K.Cache(F, kind, kv_heads, dim, 16, -(-length // 16), 5)
    call = X.Call(F, cache, heads, [new], [length], wide=wide)
    ref = call.reference()
    if kind == 0:
        cache.t[1].fill_(float("nan"))
    else:
        cache.scales[1].fill_(255)
    out, lse = call.run()
    assert np.all(np.isnan(out))
    X.check(np.zeros_like(out), lse, (np.zeros_like(out), *ref[1:]))


def _spread_cache(F, kind, kv_heads, dim, page, n_pages, form, seed, special=()):
    """A cache whose values' scales are far apart: from block to block of a row, from token to token, over the format's whole
    range, or only those of the `special` slots far above all others."""
    cache = K.Cache(F, kind, kv_heads, dim, page, n_pages, seed)
    rng = np.random.default_rng(seed + 100)
    shape = (n_pages, kv_heads, page, dim // 32)
    top = 134 if kind == 1 else 140  # the largest scale code of the format
    if form == "blocks":
        code = np.broadcast_to(np.array([top, top - 30, top - 60, 27, top - 15, 60, top - 25, top - 1])[: dim // 32], shape)
    elif form == "tokens":
        code = np.where(rng.random(shape[:3]) < 0.03, top, top - 32)[..., None] + np.zeros(shape, dtype=int)
    elif form == "range":
        code = rng.integers(27, top + 1, shape)
    else:
        code = np.full(shape, top - 35)
        for s in special:
            code[s // page, :, s % page] = top
    scale = np.ascontiguousarray(code).astype(np.uint8)
    cache.scales[1].copy_(torch.from_numpy(scale))
    cache.value[1] = K.stands_for(cache.t[1].cpu().numpy(), scale, kind)
    return cache


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("form", ["blocks", "tokens", "range"])
@pytest.mark.parametrize("new,length,wide", [(1, 1, 0), (1, 500, 0), (5, 300, 0), (70, 200, WIDE)])
def test_values_of_small_scale_are_kept_beside_large_ones(F, kind, heads, kv_heads, dim, form, new, length, wide):
    """Column by column, with single tokens (one row tile), a few (two, where there are such) and a chunk.  The smallest scale,
    2^-100, times MXFP4's smallest element and a probability is near the end of FP32's range: `floor` as kvexact.py says."""
    cache = _spread_cache(F, kind, kv_heads, dim, 16, -(-length // 16) + 1, form, dim + new)
    X.Call(F, cache, heads, [new], [length], wide=wide).check(floor=length * 2.0 ** -104 * (2.0 ** -100 * 6))


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("new,length,window,wide", [(6, 200, 0, 0), (6, 200, 40, 0), (70, 200, 0, WIDE), (70, 200, 40, 0)])
def test_large_values_that_a_row_does_not_see_change_nothing(F, kind, heads, kv_heads, dim, new, length, window, wide):
    """The last new token, and the one before the last row's window, have values 2^35 times as large as the others: rows that
    do not see them, column by column, and rows that do."""
    at = [length - 1] + ([length - window - 1] if window else [])
    cache = _spread_cache(F, kind, kv_heads, dim, 16, -(-length // 16), "special", new, at)
    table = np.arange(-(-length // 16), dtype=np.int32)[None]
    X.Call(F, cache, heads, [new], [length], table, window=window, wide=wide).check()


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("new,wide", [(1, 0), (5, 0), (70, WIDE)])
def test_a_large_value_of_next_to_no_probability_takes_nothing_away(F, kind, heads, kv_heads, dim, new, wide):
    """One token of values near the format's largest, whose probability is about 2^-60, beside tokens of values 2^15 smaller:
    it adds 2^-45 of them, and their own sums keep every term."""
    length, at = 260, 77
    cache = _spread_cache(F, kind, kv_heads, dim, 16, 17, "special", new, [at])
    scale = np.full((17, kv_heads, 16, dim // 32), 119, dtype=np.uint8)
    scale[at // 16, :, at % 16] = 134
    cache.scales[1].copy_(torch.from_numpy(scale))
    cache.value[1] = K.stands_for(cache.t[1].cpu().numpy(), scale, kind)
    table = np.arange(17, dtype=np.int32)[None]
    call = X.Call(F, cache, heads, [new], [length], table, wide=wide, scale=0.01)
    # every query has a part against the token's key that makes its score 60 log 2 smaller than the others'
    key = cache.value[0][at // 16, :, at % 16]                        # [kv_heads][dim]
    group = heads // kv_heads
    q = call.q.reshape(new, kv_heads, group, dim)
    need = -60 * np.log(2) / 0.01
    q = q + ((need - (q * key[:, None]).sum(-1)) / (key * key).sum(-1)[:, None])[..., None] * key[:, None]
    call.q_t.copy_(torch.from_numpy(q.reshape(new, heads, dim).astype(np.float32)).to(torch.bfloat16))
    call.q = call.q_t.double().cpu().numpy()
    call.check()


# Heads, cache heads, head width and new tokens of chunks with a window that are much work all the same.
WINDOWED = [(64, 2, 64, 600), (64, 1, 128, 400), (32, 1, 256, 400)]


@pytest.mark.parametrize("kind,copies", [(0, True), (1, True), (1, False), (2, True), (2, False)])
@pytest.mark.parametrize("heads,kv_heads,dim,new", WINDOWED + [(4, 1, 64, 4), (8, 1, 128, 3), (16, 2, 256, 1)])
@pytest.mark.parametrize("page,window", [(16, 50), (64, 50), (128, 301)])
def test_tokens_before_every_window_do_not_matter(F, kind, copies, heads, kv_heads, dim, new, page, window):
    """Keys and values of the tokens before the first row's window are no numbers, some of them in the window's first page."""
    length = new + 700
    first = length - new - window + 1  # the first token that any row sees
    pages = -(-length // page)
    cache = K.Cache(F, kind, kv_heads, dim, page, pages, 8)
    table = np.arange(pages, dtype=np.int32)[None]
    call = X.Call(F, cache, heads, [new], [length], table, window=window, copies=copies)
    ref = call.reference(lambda s, i: i < 8 or i % 37 == 0)
    assert first % page
    for j in range(first - 40, first):
        for i in (0, 1):
            if kind == 0:
                cache.t[i][j // page, :, j % page] = float("nan") if j % 3 else float("inf")
            else:
                cache.scales[i][j // page, :, j % page] = 255
    got = call.run()
    assert call.word.item() == 0
    X.check(*got, ref)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_a_slot_that_two_tokens_name_leaves_other_rows_alone(F, kind):
    """The row itself is undefined; every other one is as without the repeated slot."""
    heads, dim, page, n = 3, 128, 16, 40
    rng = np.random.default_rng(2)
    x = [torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in "kv"]
    cache = X.Cache(F, kind, *(np.zeros((4, heads, page, dim)) for _ in "kv"))
    slots = rng.permutation(4 * page)[:n]
    slots[7] = slots[31]
    on = torch.from_numpy(slots.astype(np.int32)).cuda()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    F.ft_kv_write(cache.c, *x, on, error_word=word)
    every = [torch.empty(4 * page, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    F.ft_kv_read(cache.c, torch.arange(4 * page, dtype=torch.int32, device="cuda"), *every, error_word=word)
    torch.cuda.synchronize()
    assert word.item() == 0
    for t, rows in zip(x, every):
        want = np.zeros((4 * page, heads, dim))
        a = t.double().cpu().numpy()
        if kind:
            code, scale = K.quantise(a, kind)
            a = K.stands_for(K.packed(code, kind), scale, kind)
        want[slots] = a
        others = np.arange(4 * page) != slots[7]
        assert np.array_equal(rows.double().cpu().numpy()[others], want[others])


SHAPES = [(4, 4, 64), (6, 2, 128), (7, 1, 128), (16, 2, 256), (40, 2, 64)]


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
@pytest.mark.parametrize("window", [0, 37])
def test_every_column_of_ragged_batches(F, kind, heads, kv_heads, dim, window):
    """Single tokens, drafts and short chunks side by side."""
    cache = K.Cache(F, kind, kv_heads, dim, 16, 120, 3)
    X.Call(F, cache, heads, [1, 1, 3, 1, 5, 2, 1, 40], [1, 17, 333, 64, 128, 2, 500, 260], window=window).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (3, 1, 64), (4, 2, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_every_column_of_chunks(F, kind, heads, kv_heads, dim, causal):
    cache = K.Cache(F, kind, kv_heads, dim, 64, 30, 3)
    X.Call(F, cache, heads, [129, 70, 200], [129, 500, 777], causal=causal, wide=WIDE).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,new,wide", [
    (4, 1, 64, 1, 0), (8, 1, 128, 1, 0), (8, 1, 128, 4, 0), (16, 2, 256, 1, 0), (4, 1, 64, 40, WIDE), (8, 1, 128, 40, WIDE),
    (4, 2, 256, 70, WIDE), (32, 1, 128, 40, WIDE)])
@pytest.mark.parametrize("length", [4001, 9003])
def test_every_tile_of_a_long_cache_counts_once(F, kind, heads, kv_heads, dim, new, wide, length):
    """One token of every 32 has an even share of nearly all of the probability, and a one in the column of its run of tokens: a
    lost, doubled or wrongly weighted tile of any part shows in the columns that few tokens fill."""
    page = 32
    pages = -(-length // page)
    rng = np.random.default_rng(length)
    k, v = rng.standard_normal((pages, kv_heads, page, dim)) * 0.01, np.zeros((pages, kv_heads, page, dim))
    per = -(-pages // dim)  # marked tokens of a column
    for j, off in enumerate(rng.integers(0, page, pages)):
        k[j, :, off] = 1.0
        v[j, :, off, j // per] = 1.0
    table = rng.permutation(pages).astype(np.int32)
    back = np.argsort(table)
    cache, table = X.Cache(F, kind, k[back], v[back]), table[None]
    q = np.ones((new, heads, dim)) + rng.standard_normal((new, heads, dim)) * 0.01
    keep = {0, new // 2, new - 1}
    call = X.Call(F, cache, heads, [new], [length], table, scale=24 / dim, q=q, wide=wide)
    call.check(rows=lambda s, i: i in keep)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(16, 2, 256, 128), (32, 4, 128, 64), (24, 8, 64, 16)])
def test_every_column_of_both_kernels_agrees(F, kind, heads, kv_heads, dim, page):
    """The kernels for few and for many rows over several thousand tokens, each within its bound of the definition."""
    cache = K.Cache(F, kind, kv_heads, dim, page, 6001 // page + 400 // page + 2, 3)
    keep = {(0, 0), (0, 250), (0, 499), (1, 0), (1, 32)}
    few, many = (X.Call(F, cache, heads, [500, 33], [6001, 400], max_new=m) for m in (1, 500))
    ref = few.reference(lambda s, i: (s, i) in keep)
    for call in (few, many):
        X.check(*call.run(), ref)
        assert call.word.item() == 0


@pytest.mark.parametrize("kind,heads,kv_heads,dim,new,lens,wide", [
    (0, 8, 1, 128, [1, 1], [4000, 30], 0), (1, 8, 1, 128, [1, 5], [4000, 30], 0), (2, 16, 2, 256, [3, 1], [700, 90], 0),
    (0, 8, 1, 128, [60, 1], [900, 50], WIDE), (1, 32, 1, 128, [60, 1], [900, 50], WIDE), (2, 16, 2, 256, [40, 3], [300, 20], WIDE)])
def test_only_the_counters_of_a_workspace_need_to_be_cleared(F, kind, heads, kv_heads, dim, new, lens, wide):
    """Bytes that are no numbers everywhere else: the same bits, also on the second call."""
    cache = K.Cache(F, kind, kv_heads, dim, 16, sum(-(-n // 16) for n in lens), 6)
    call = X.Call(F, cache, heads, new, lens, wide=wide)
    want = call.run()
    call.ws.fill_(0xFF)
    call.ws[:F.FT_ATTN_CLEAR_BYTES].zero_()
    for _ in range(2):
        call.out.fill_(77.0)
        assert all(np.array_equal(a, b) for a, b in zip(call.run(), want))
    assert call.word.item() == 0 and call.ws[:F.FT_ATTN_CLEAR_BYTES].max().item() == 0


# Batches whose rows see different tokens of their blocks: few rows (one and two row tiles) and many.
PARTLY = [(4, 2, 64, 6, 300, 0), (8, 1, 128, 4, 300, 0), (16, 2, 256, 3, 300, 0), (4, 2, 64, 20, 300, 7), (8, 1, 128, 9, 300, 5),
          (4, 1, 64, 200, 500, 0), (8, 1, 128, 100, 500, 0), (16, 2, 256, 70, 400, 0), (1, 1, 128, 300, 700, 0),
          (64, 2, 64, 600, 1000, 40), (64, 1, 128, 400, 900, 130), (32, 1, 256, 400, 600, 3)]


@pytest.mark.parametrize("kind,copies", [(0, True), (1, True), (1, False), (2, True), (2, False)])
@pytest.mark.parametrize("heads,kv_heads,dim,new,length,window", PARTLY)
def test_single_elements_that_are_not_finite(F, kind, copies, heads, kv_heads, dim, new, length, window):
    """Some elements (quantised: 1x32 blocks) of some new tokens' values are infinite or NaN.  Rows that do not see such a
    token are as if it were not there; rows that do have the sum that IEEE gives in those columns, and the others as always."""
    rng = np.random.default_rng(new + dim)
    pages = -(-length // 32)
    cache = K.Cache(F, kind, kv_heads, dim, 32, pages, 9)
    table = np.arange(pages, dtype=np.int32)[None]
    call = X.Call(F, cache, heads, [new], [length], table, window=window, wide=0 if window or new < 30 else WIDE, copies=copies)
    keep = {0, 1, new // 2, new - 2, new - 1} | set(range(0, new, max(1, new // 23)))
    clean = cache.value[1].copy()
    extra = np.zeros_like(clean)                       # what is not finite
    for j in rng.choice(np.arange(length - new, length), min(new, 9), replace=False):
        h, col = int(rng.integers(kv_heads)), int(rng.integers(dim))
        at = (j // 32, h, j % 32)
        if kind == 0:
            value = [np.inf, -np.inf, np.nan][int(rng.integers(3))]
            cache.t[1][at[0], at[1], at[2], col] = value
            extra[at][col], clean[at][col] = value, 0.0
        else:
            block = slice(col // 32 * 32, col // 32 * 32 + 32)
            cache.scales[1][at[0], at[1], at[2], col // 32] = 255
            extra[at][block], clean[at][block] = np.nan, 0.0
    cache.value[1] = clean
    ref = call.reference(lambda s, i: i in keep)
    got = call.run()
    assert call.word.item() == 0
    bad = np.zeros_like(ref[0])                        # what the rows see of it, summed
    group = heads // kv_heads
    for i in keep:
        p = length - new + i
        lo = max(0, p - window + 1) if window else 0
        for h in range(kv_heads):
            with np.errstate(invalid="ignore"):
                bad[i, h * group:(h + 1) * group] = extra[:, h].reshape(-1, dim)[lo:p + 1].sum(0)
    some = np.array([i in keep for i in range(new)])[:, None, None] & (bad != 0)
    assert some.any()
    assert np.array_equal(got[0][some], bad[some], equal_nan=True)
    X.check(np.where(some, ref[0], got[0]), got[1], ref)


@pytest.mark.parametrize("kind", [0, 1])
def test_a_long_chunk_whose_last_value_is_not_finite(F, kind):
    """Every row but the last is as it should be, in about the time that the chunk takes anyway."""
    heads, kv_heads, dim, length, page = 8, 4, 128, 24576, 64
    pages = length // page
    cache = K.Cache(F, kind, kv_heads, dim, page, pages, 2)
    table = np.random.default_rng(1).permutation(pages).astype(np.int32)[None]
    call = X.Call(F, cache, heads, [length], [length], table)
    keep = {5, 4000, length - 100, length - 3, length - 2}
    ref = call.reference(lambda s, i: i in keep)
    call.run()
    took = []
    for put in (False, True):
        if put and kind == 0:
            cache.t[1][table[0, -1], :, page - 1] = float("nan")
        elif put:
            cache.scales[1][table[0, -1], :, page - 1] = 255
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        got = call.run()
        b.record()
        b.synchronize()
        took.append(a.elapsed_time(b))
        assert call.word.item() == 0
        X.check(*got, ref)
    assert np.all(np.isnan(got[0][-1])) and np.all(np.isfinite(got[0][:-1])) and np.all(np.isfinite(got[1]))
    assert took[1] < 5 * took[0] + 10, took
