"""The column bounds of kvexact.py find what they are there for: mistakes planted in results that are right otherwise."""
import numpy as np
import pytest

import kvexact as X


class Rows:
    """A cache on the host: [page][head][token][dim] float64."""

    def __init__(self, k, v):
        self.value, (_, self.heads, self.page, self.dim) = (k, v), k.shape

    def rows(self, which, pages, head, length):
        return self.value[which][pages, head].reshape(-1, self.dim)[:length]


def _case(marked):
    rng = np.random.default_rng(1)
    pages, page, dim, heads = 125, 32, 64, 4
    k, v = rng.standard_normal((2, pages, 1, page, dim))
    if marked:  # one token of a page has an even share of the probability, and a one in a column of few
        k, v = k * 0.01, v * 0
        for j, off in enumerate(rng.integers(0, page, pages)):
            k[j, :, off] = 1.0
            v[j, :, off, j // 2] = 1.0
    q = np.ones((1, heads, dim)) if marked else rng.standard_normal((1, heads, dim))
    cache, table = Rows(k, v), np.arange(pages)[None]
    ref = X.attention(cache, q, [0, 1], [pages * page - 7], table, 24 / dim if marked else dim ** -0.5)
    return cache, q, table, ref


def _to_bf16(x):
    """Rounded to 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256), e - 8)


@pytest.mark.parametrize("marked", [False, True])
def test_rounded_results_pass(marked):
    *_, ref = _case(marked)
    X.check(_to_bf16(ref[0]), ref[2].astype(np.float32).astype(float), ref)


@pytest.mark.parametrize("mistake", ["a lost tile", "a tile counted twice", "a tile of half the weight", "a tile of other values"])
def test_a_wrong_tile_does_not_pass(mistake):
    """64 of 3993 tokens, in the product with the values alone (lse as it should be)."""
    cache, q, table, ref = _case(True)
    k, v = (cache.rows(i, table[0], 0, 3993) for i in (0, 1))
    p = np.exp(24 / cache.dim * (q[0] @ k.T) - ref[2][0][:, None])
    w = p.copy()
    w[:, 1280:1344] *= {"a lost tile": 0, "a tile counted twice": 2, "a tile of half the weight": 0.5}.get(mistake, 1)
    if mistake == "a tile of other values":
        v = v.copy()
        v[1280:1344] = v[640:704]
    with pytest.raises(AssertionError):
        X.check(_to_bf16((w @ v)[None]), ref[2], ref)


def test_zeros_do_not_pass():
    *_, ref = _case(False)
    with pytest.raises(AssertionError):
        X.check(ref[0] * 0, ref[2], ref)
    bad = ref[0].copy()
    bad[0, 2, 5:9] = 0
    with pytest.raises(AssertionError):
        X.check(bad, ref[2], ref)
