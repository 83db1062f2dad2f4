"""Attention over the paged cache beyond the ordinary: every kernel that a batch's size can choose (a table with room for
many more pages says that there may be much to do, so the kernel for many rows runs on lengths that a reference can follow),
copies of quantised pages that fit their room or do not, scores' scales of any sign, bad pages, a stream of its own, and
offsets beyond 32 bits.  Tolerances are those of test_gpu_kv.py, unless a test says otherwise."""
import numpy as np
import pytest
import torch

import kvharness as K
from test_gpu_kv import F, Batch  # noqa: F401  (F is a fixture)

pytestmark = pytest.mark.gpu

STAGING = 512 << 20  # bytes of the workspace's part for decoded pages


def widen(b, pages, max_new, small=False):
    """The batch again, its table with `pages` more entries a sequence (naming no page); small: without room for copies."""
    table = torch.cat([b.dev[2], torch.full((len(b.lens), pages), 2 ** 31 - 1, dtype=torch.int32, device="cuda")], 1)
    ws = b.ws[: b.ws.numel() - STAGING] if small else b.ws
    b.dev[2] = table
    b.args = b.F.make_attn_args(b.heads, max_new, b.q_t, *b.dev, b.out, ws, scale=b.scale, window=b.window, causal=b.causal,
                                lse=b.lse, error_word=b.word)
    return b


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (3, 1, 64), (4, 2, 256)])
@pytest.mark.parametrize("new,length", [(129, 129), (200, 777), (64, 1000), (23, 40)])
def test_chunks_with_room_for_long_ones(F, kind, heads, kv_heads, dim, new, length):
    widen(Batch(F, kind, heads, kv_heads, dim, 32, new=[new], lens=[length]), 20000, 1000).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,new", [(64, 8, 64, 600), (64, 8, 128, 400), (32, 2, 256, 400)])
@pytest.mark.parametrize("window,causal", [(1, True), (40, True), (300, False)])
def test_windows_of_many_rows(F, kind, heads, kv_heads, dim, new, window, causal):
    """Windows narrower than a tile and wider; without `causal`, rows see what is behind them to the end."""
    b = Batch(F, kind, heads, kv_heads, dim, 64, new=[new, 3, 1], lens=[new + 333, 500, 1], window=window, causal=causal)
    widen(b, 40000, new).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (7, 1, 128), (8, 4, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_batches_with_room_for_long_ones(F, kind, heads, kv_heads, dim, causal):
    """Rows that see nothing, lengths of zero, sequences without new tokens, pages that end inside a tile."""
    b = Batch(F, kind, heads, kv_heads, dim, 16, new=[1, 70, 0, 5, 3, 1], lens=[300, 70, 45, 5, 0, 1],
              causal=causal, extra_rows=2, wide=True)
    widen(b, 40000, 1000).check()


FORMS = ["copied", "table too wide", "no workspace"]


@pytest.mark.parametrize("dim,heads,kv_heads,kind,form,window", [
    (d, h, kvh, kind, form, 0) for d, h, kvh in ((64, 32, 2), (128, 32, 2), (256, 16, 1)) for kind in (1, 2) for form in FORMS
] + [(256, 16, 1, 1, "copied", 6900), (128, 32, 2, 2, "table too wide", 6900), (64, 32, 2, 1, "no workspace", 6900)])
def test_many_rows_over_a_quantised_cache(F, kind, dim, heads, kv_heads, form, window):
    """1024 rows of a head and more: pages are decoded once, with and without a table that could name more pages than there
    is room for, or, without the workspace for it, where they are read."""
    b = Batch(F, kind, heads, kv_heads, dim, 16, new=[66, 1, 0, 7], lens=[7000 if window else 200, 90, 33, 7], window=window)
    room = STAGING // 2 // (kv_heads * 16 * dim * 2) // 4  # pages of a sequence, four of which fill it
    widen(b, room + 1 if form == "table too wide" else room // 2, 66, small=form == "no workspace")
    b.check()
    first = b.out.clone()
    b.check()
    assert torch.equal(first, b.out)


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("repeats", [1, 65])
def test_copies_that_have_room_and_that_have_none(F, kind, repeats):
    """A table wider than the room for copies, of few pages or of more than there is room for: 64 pages again and again.
    Every token sees all of them (not causal), so out is that over 64 pages and lse is log(repeats) more.  Sums of up to
    66560 terms are rounded at most that many times: 66560 * 2^-24 of the values, of out and lse, besides the other bounds."""
    heads, kv_heads, dim, page, new = 128, 8, 256, 16, 64
    rng = np.random.default_rng(5)
    c = K.Cache(F, kind, kv_heads, dim, page, 64, 3)
    length = 64 * page * repeats
    table = np.full((1, 64 * 65 + 1), -1, dtype=np.int32)
    table[0, :64 * repeats] = np.tile(np.arange(64), repeats)
    q = torch.from_numpy(rng.standard_normal((new, heads, dim)).astype(np.float32)).to(torch.bfloat16).cuda()
    out, lse = torch.empty_like(q), torch.empty(new, heads, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(F.ft_attn_workspace(heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
    dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [length])] + [torch.from_numpy(table).cuda()]
    assert table.shape[1] * kv_heads * page * dim * 2 > STAGING // 2
    a = F.make_attn_args(heads, new, q, *dev, out, ws, scale=1 / 16, causal=False, lse=lse, error_word=word)
    F.ft_attn(c.c, a)
    torch.cuda.synchronize()
    assert word.item() == 0
    got, got_lse, q64 = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for h in range(heads):
        k, v = (c.rows(i, np.arange(64), h // 16, 64 * page) for i in (0, 1))
        z = q64[:, h] @ k.T / 16
        top = z.max(1, keepdims=True)
        e = np.exp(z - top)
        ref, ref_lse = (e / e.sum(1, keepdims=True)) @ v, top[:, 0] + np.log(e.sum(1)) + np.log(repeats)
        d = 1.01 * (dim + 4) * 2.0 ** -24 / 16 * (np.abs(q64[:, h]) @ np.abs(k).T).max() + 66560 * 2.0 ** -24
        assert np.all(np.abs(got[:, h] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * d + 2.0 ** -20) * np.abs(v).max())
        assert np.all(np.abs(got_lse[:, h] - ref_lse) <= d + 2.0 ** -20 * (1 + np.abs(ref_lse)))


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("dim,new", [(64, 3), (128, 1), (256, 2), (64, 70), (128, 40), (256, 80)])
def test_scales_of_any_sign(F, kind, scale, dim, new):
    b = Batch(F, kind, 6, 2, dim, 16, new=[new, 1], lens=[new + 90, 17], scale=scale)
    widen(b, 40000 if new > 3 else 0, 1000 if new > 3 else new).check()


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [70, 1100])
def test_bad_pages_in_a_chunk_are_reported(F, kind, dim, rows):
    """A page beyond the cache, or below it, counts as rows of zeros; other sequences are as they were."""
    new = rows // 16 + 1
    b = widen(Batch(F, kind, 32, 2, dim, 16, new=[new, new], lens=[new + 60, new + 60], stale_nan=False), 40000, new)
    good, _ = b.run()
    good = good.copy()
    n = int(b.q_start[1])
    for bad in (b.cache.n_pages, -1, -2 ** 31):
        b.word.zero_()
        b.dev[2][0, 1] = bad
        out, lse = b.run()
        assert b.word.item() == F.FT_DEVERR_BAD_INDEX and np.array_equal(out[n:], good[n:])
        # the same with a page of zeros in that place
        zero = [t.clone() for t in b.cache.t]
        page = b.table[0, 1]
        for t in zero:
            t[page] = 0
        c = F.make_kv_cache(kind, 2, dim, 16, b.cache.n_pages, *zero, *b.cache.scales)
        b.dev[2][0, 1] = int(page)
        b.word.zero_()
        F.ft_attn(c, b.args)
        torch.cuda.synchronize()
        assert b.word.item() == 0
        assert np.array_equal(b.out.double().cpu().numpy()[:n], out[:n]) and np.array_equal(b.lse.double().cpu().numpy()[:n], lse[:n])


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim,new,length,window", [
    (4, 1, 64, 140, 400, 0), (8, 1, 128, 60, 200, 0), (16, 2, 256, 40, 130, 0), (8, 1, 128, 300, 1500, 0), (64, 8, 128, 400, 900, 50)])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_values_that_many_rows_do_not_see_do_not_matter(F, kind, heads, kv_heads, dim, new, length, window, value):
    """A token within the chunk whose keys and values are not finite: rows that do not see it are as if it were not there,
    rows that see it are NaN."""
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
    out, lse = widen(b, 20000, new).check(rows=lambda s, i: not sees(s, i))
    seeing = [i for i in range(new) if sees(0, i)]
    assert seeing and np.all(np.isnan(out[seeing])) and np.all(np.isnan(lse[seeing]))


def test_work_goes_to_the_given_stream(F):
    """Inputs that are put in place on the stream, late, are the ones that are used."""
    s = torch.cuda.Stream()
    for kind, new in ((0, 1), (1, 80)):
        b = widen(Batch(F, kind, 32, 2, 128, 16, new=[new], lens=[200]), 40000 if new > 1 else 0, new)
        want, _ = b.run()
        q = b.q_t.clone()
        b.q_t.zero_()
        b.out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            b.q_t.copy_(q)
        F.ft_attn(b.cache.c, b.args, stream=s.cuda_stream)
        s.synchronize()
        assert np.array_equal(b.out.double().cpu().numpy(), want)


def test_a_workspace_that_is_too_small_is_refused(F):
    b = Batch(F, 1, 8, 2, 128, 16, new=[1], lens=[40])
    b.out.fill_(7.0)
    for n in (64, 256, b.ws.numel() - STAGING - 8192):
        a = F.make_attn_args(8, 1, b.q_t, *b.dev, b.out, b.ws[:n], scale=b.scale)
        with pytest.raises(F.FtError) as e:
            F.ft_attn(b.cache.c, a)
        assert e.value.status == F.FT_ERR_CAPACITY
    torch.cuda.synchronize()
    assert torch.all(b.out == 7.0)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("new", [1, 5, 200])
def test_pages_beyond_four_gigabytes(F, kind, new):
    """The same rows in the last pages of a cache of more than 2^32 bytes as in a small cache: the same bits, written, read
    and attended to."""
    heads, dim, page, n = 8, 128, 64, 13
    per = heads * page * dim * (2 if kind == 0 else 1 if kind == 1 else 0.5)
    n_pages = int(4.5 * 2 ** 30 / per)
    rng = np.random.default_rng(1)
    length = n * page - 5
    k, v = (torch.from_numpy(rng.standard_normal((length, heads, dim)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((new, 64, dim)).astype(np.float32)).to(torch.bfloat16).cuda()
    ws = torch.zeros(F.ft_attn_workspace(64, heads, dim), dtype=torch.uint8, device="cuda")
    got = []
    for total, first in ((n, 0), (n_pages, n_pages - n)):
        width = {0: dim, 1: dim, 2: dim // 2}[kind]
        kc, vc = (torch.empty(total, heads, page, width, dtype=torch.bfloat16 if kind == 0 else torch.uint8, device="cuda") for _ in range(2))
        scales = [torch.empty(total, heads, page, dim // 32, dtype=torch.uint8, device="cuda") if kind else None for _ in range(2)]
        c = F.make_kv_cache(kind, heads, dim, page, total, kc, vc, *scales)
        slots = torch.arange(length, dtype=torch.int32, device="cuda") + first * page
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        F.ft_kv_write(c, k, v, slots, error_word=word)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        F.ft_kv_read(c, slots, ko, vo, error_word=word)
        out, lse = torch.empty_like(q), torch.empty(new, 64, device="cuda")
        dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [length])]
        table = torch.full((1, 20000), -1, dtype=torch.int32, device="cuda")
        table[0, :n] = torch.arange(n, device="cuda") + first
        F.ft_attn(c, F.make_attn_args(64, new, q, *dev, table, out, ws, scale=0.1, lse=lse, error_word=word))
        torch.cuda.synchronize()
        assert word.item() == 0
        got.append((ko, vo, out, lse))
        del kc, vc, scales, c
    for a, b in zip(*got):
        assert torch.equal(a, b)
    if kind == 0:
        assert torch.equal(got[0][0], k) and torch.equal(got[0][1], v)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("heads,kv_heads,dim", [(24, 8, 64), (32, 4, 128), (16, 2, 256)])
@pytest.mark.parametrize("window", [0, 700])
def test_batches_of_single_tokens_and_chunks(F, kind, heads, kv_heads, dim, window):
    """Sequences of few and of many rows side by side, with tables that name enough to read for a launch each."""
    new, lens = [1, 90, 2, 1, 0, 130, 1, 3], [1000, 90, 2, 777, 50, 400, 1, 0]
    b = Batch(F, kind, heads, kv_heads, dim, 64, new=new, lens=lens, window=window, extra_rows=3)
    widen(b, 1 << 14, 130).check()
    first = b.out.clone()
    b.check()
    assert torch.equal(first, b.out)
