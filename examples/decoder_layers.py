"""Decoder layers with attention over a paged cache and experts from the slot pool.

    python examples/decoder_layers.py [--cache bf16|mxfp8|mxfp4] [--prompt N] [--tokens N]

Every layer: a projection to queries, keys and values; ft_kv_write puts the new tokens' keys and
values into the layer's pages; ft_attn attends over them; an output projection; then the MoE half,
routed from the hidden states (ft_moe_prefill_chunk_hidden for chunks, ft_moe_decode_step_hidden for
single tokens).  The prompt goes through in chunks, the tokens after it one by one.  Weights are
random, and the "next token" is the last hidden state again, normalised: this shows how the calls go
together, not a model.  Projections and norms are plain torch operations.
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
from serving_router_top_dedupe_gb300 import ftmoe as F  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 4, 2, 64, 16
KINDS = {"bf16": F.FT_KV_BF16, "mxfp8": F.FT_KV_MXFP8, "mxfp4": F.FT_KV_MXFP4}


def norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Layers:
    """A stack of layers with the cache of one session."""

    def __init__(self, cache="bf16", max_tokens=512, chunk=64, seed=1):
        w = synth.tiny()
        self.w, self.chunk, self.length = w, chunk, 0
        self.banks = synth.ExpertPool(w).routed_banks()
        # Both halves of a layer, and torch's operations between them, go to one stream.  It has to be named: the legacy
        # default stream is NULL, for which the MoE half would make a stream of its own that nothing here waits for.
        self.on = torch.cuda.Stream()
        self.stream = self.on.cuda_stream
        # B_H below B_P: every expert that misses the slot pool is filled, none is left to the host
        cfg = F.make_config(w.n_layers, w.hidden, w.inter, w.n_experts, w.top_k, False, F.FT_W_BF16, 1, 2 * w.n_experts,
                            50.0, 40.0, max_prefill_tokens=chunk, compute_stream=self.stream)
        self.moe = F.ft_moe_init(cfg, self.banks)
        F.ft_moe_set_router(self.moe, synth.router_weights(w))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n_in, n_out):
            return (torch.randn(n_in, n_out, generator=g, device="cuda") / math.sqrt(n_in)).to(torch.bfloat16)

        self.qkv = [weight(w.hidden, (HEADS + 2 * KV_HEADS) * DIM) for _ in range(w.n_layers)]
        self.proj = [weight(HEADS * DIM, w.hidden) for _ in range(w.n_layers)]
        pages = -(-max_tokens // PAGE)
        kind = KINDS[cache]
        per = {F.FT_KV_BF16: DIM, F.FT_KV_MXFP8: DIM, F.FT_KV_MXFP4: DIM // 2}[kind]
        dt = torch.bfloat16 if kind == F.FT_KV_BF16 else torch.uint8
        self.caches = []
        for _ in range(w.n_layers):
            k, v = (torch.zeros(pages, KV_HEADS, PAGE, per, dtype=dt, device="cuda") for _ in "kv")
            sc = [torch.zeros(pages, KV_HEADS, PAGE, DIM // 32, dtype=torch.uint8, device="cuda") for _ in "kv"] if kind else [None] * 2
            self.caches.append(F.make_kv_cache(kind, KV_HEADS, DIM, PAGE, pages, k, v, *sc))
        # pages in an order of their own, as a session gets them from a pool
        self.table = torch.randperm(pages, generator=g, device="cuda").int()[None].contiguous()
        # chunks have fewer than 1024 rows of a cache head here: no room for decoded pages
        self.workspace = torch.empty(F.ft_attn_workspace(HEADS, KV_HEADS, DIM) - F.FT_ATTN_COPY_BYTES, dtype=torch.uint8, device="cuda")
        self.workspace[:F.FT_ATTN_CLEAR_BYTES].zero_()
        self.kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, x, keep=None):
        """Hidden states [n][hidden] BF16 of the next n tokens -> theirs after the layers, for the current stream.  keep: a
        list that gets every layer's (queries, attention output)."""
        caller = torch.cuda.current_stream()
        self.on.wait_stream(caller)
        with torch.cuda.stream(self.on):
            x = self._forward(x, keep)
        caller.wait_stream(self.on)
        return x

    def _forward(self, x, keep):
        n, w = x.shape[0], self.w
        at = torch.arange(self.length, self.length + n, dtype=torch.int32, device="cuda")
        slots = self.table[0, (at // PAGE).long()] * PAGE + at % PAGE
        self.length += n
        self.kv_len.fill_(self.length)
        q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for layer in range(w.n_layers):
            qkv = (norm(x) @ self.qkv[layer]).view(n, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            cache, attn = self.caches[layer], torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
            F.ft_kv_write(cache, k, v, slots, error_word=self.error, stream=self.stream)
            args = F.make_attn_args(HEADS, n, q, q_start, self.kv_len, self.table, attn, self.workspace,
                                    scale=1 / math.sqrt(DIM), error_word=self.error)
            F.ft_attn(cache, args, stream=self.stream)
            if keep is not None:
                keep.append((q.clone(), attn.clone()))
            x = x + attn.view(n, -1) @ self.proj[layer]
            h, out = norm(x).contiguous(), torch.empty(n, w.hidden, device="cuda")
            if n == 1:
                F.ft_moe_decode_step_hidden(self.moe, layer, 1, h, None, out)
            else:
                F.ft_moe_prefill_chunk_hidden(self.moe, layer, n, h, out)
            x = x + out.to(torch.bfloat16)
        return x

    def prompt(self, x, keep=None):
        """A whole prompt in chunks; the last token's hidden state."""
        for i in range(0, x.shape[0], self.chunk):
            y = self.forward(x[i:i + self.chunk], keep)
        return y[-1:]

    def close(self):
        F.ft_moe_destroy(self.moe)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--cache", choices=list(KINDS), default="mxfp8")
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    m = Layers(a.cache, max_tokens=a.prompt + a.tokens)
    try:
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        x = m.prompt(torch.randn(a.prompt, m.w.hidden, generator=g, device="cuda").to(torch.bfloat16))
        for _ in range(a.tokens):
            x = m.forward(norm(x))
        torch.cuda.synchronize()
        st = F.ft_moe_get_stats(m.moe)
        assert m.error.item() == 0 and st.error_word == 0 and bool(torch.isfinite(x).all())
        print(f"{a.prompt} prompt tokens in chunks of {m.chunk}, {a.tokens} decoded, {a.cache} cache of {m.length} tokens; "
              f"experts: {st.hits} hits, {st.fills} fills; |x| = {np.sqrt(float(x.float().square().mean())):.3f}")
    finally:
        m.close()


if __name__ == "__main__":
    main()
