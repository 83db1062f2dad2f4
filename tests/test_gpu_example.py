"""The example's decoder layers: attention over the paged cache and experts from the slot pool, in one session."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layers", os.path.join(ROOT, "examples", "decoder_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ["bf16", "mxfp8", "mxfp4"])
def test_layers_attend_to_what_the_cache_holds(example, cache):
    """A prompt in chunks and decoded tokens: every attention output against 64-bit attention over the keys and values that
    reading the cache back gives (the chunk's and the single tokens' kernels, both behind their writes in one stream).
    Tolerance as in test_gpu_kv.py: BF16's rounding of the probabilities and of the output."""
    E, F = example, example.F
    m = E.Layers(cache, max_tokens=150, chunk=48)
    try:
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        kept = []
        x = m.prompt(torch.randn(100, m.w.hidden, generator=g, device="cuda").to(torch.bfloat16), kept)
        for _ in range(5):
            x = m.forward(E.norm(x), kept)
        torch.cuda.synchronize()
        assert m.error.item() == 0 and F.ft_moe_get_stats(m.moe).error_word == 0 and torch.isfinite(x).all()
        n, L = m.length, m.w.n_layers
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = m.table[0, (at // E.PAGE).long()] * E.PAGE + at % E.PAGE
        for layer in range(L):
            k, v = (torch.empty(n, E.KV_HEADS, E.DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv")
            F.ft_kv_read(m.caches[layer], slots, k, v)
            q = torch.cat([a for a, _ in kept[layer::L]]).double().cpu().numpy()
            out = torch.cat([b for _, b in kept[layer::L]]).double().cpu().numpy()
            k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
            assert len(q) == n
            for h in range(E.HEADS):
                kk, vv = k[:, h * E.KV_HEADS // E.HEADS], v[:, h * E.KV_HEADS // E.HEADS]
                z = q[:, h] @ kk.T / math.sqrt(E.DIM)
                z[np.triu_indices(n, 1)] = -np.inf
                p = np.exp(z - z.max(-1, keepdims=True))
                ref = p @ vv / p.sum(-1, keepdims=True)
                d = 1.01 * (E.DIM + 4) * 2.0 ** -24 * np.max(np.abs(q[:, h]) @ np.abs(kk).T) / math.sqrt(E.DIM)
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * d + 2.0 ** -20) * np.abs(vv).max()
                assert np.all(np.abs(out[:, h] - ref) <= tol)
    finally:
        m.close()
