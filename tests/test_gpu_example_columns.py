"""The example's decoder layers again, every column of every attention output within the bound of kvexact.py."""
import math

import numpy as np
import pytest
import torch

import kvexact as X
from test_gpu_example import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


class Rows:
    def __init__(self, k, v):
        self.value, self.heads, self.page, self.dim = (k, v), k.shape[1], len(k), k.shape[2]

    def rows(self, which, pages, head, length):
        return self.value[which][:length, head]


@pytest.mark.parametrize("cache", ["bf16", "mxfp8", "mxfp4"])
def test_every_column_of_the_layers_attention(example, cache):  # noqa: F811
    E, F = example, example.F
    m = E.Layers(cache, max_tokens=220, chunk=64)
    try:
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        kept = []
        x = m.prompt(torch.randn(200, m.w.hidden, generator=g, device="cuda").to(torch.bfloat16), kept)
        for _ in range(6):
            x = m.forward(E.norm(x), kept)
        torch.cuda.synchronize()
        assert m.error.item() == 0
        n = m.length
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = m.table[0, (at // E.PAGE).long()] * E.PAGE + at % E.PAGE
        for layer in range(m.w.n_layers):
            k, v = (torch.empty(n, E.KV_HEADS, E.DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv")
            F.ft_kv_read(m.caches[layer], slots, k, v)
            q, out = (torch.cat([pair[i] for pair in kept[layer::m.w.n_layers]]).double().cpu().numpy() for i in (0, 1))
            ref = X.attention(Rows(k.double().cpu().numpy(), v.double().cpu().numpy()), q, [0, n], [n], np.zeros((1, 1), dtype=int),
                              1 / math.sqrt(E.DIM))
            X.check(out, ref[2], ref)
    finally:
        m.close()
