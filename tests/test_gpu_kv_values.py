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
