"""Cases of the paged key/value cache and of the attention that reads it.

Three operators:

  write  the new tokens' keys and values go into pages of the cache, quantised on the way where the
         cache is held in 8 or 4 bits, and are read back as the attention will see them
  read   cached tokens are gathered from their pages into dense BF16 rows
  attn   each new token of a batch of sequences attends to its sequence's cached tokens

A cache holds pages of `page` tokens; a page is [kv_heads][page][head_dim] for the keys and again for
the values.  Types: "bf16"; "mxfp8" (E4M3 elements) and "mxfp4" (E2M1 elements, two to a byte, element
2j in the low nibble), both with one E8M0 scale for 32 neighbouring elements of a row.

Quantisation of a block x[0..31] (a = max |x|):
  e = the smallest integer with a <= m * 2^e, clamped to [-100, c]    (mxfp8: m = 448, c = 7; mxfp4: m = 6, c = 13)
  element = x * 2^-e rounded to the element type, to nearest, ties to even, limited to +-m; scale code = e + 127
A cached element stands for element * 2^e, which BF16 holds exactly.

Attention of row i of a sequence with n new tokens and L cached ones (the new ones among them):
  p = L - n + i;  j attends if j <= p and (no window or j > p - window)
  s_j = scale * q_i . k_j;  lse = log sum_j exp(s_j);  out = sum_j exp(s_j - lse) v_j
"""
import math

import torch

own = False

#: Query heads, heads of the cache, head width.  Generic layouts: grouped heads at the common widths, groups
#: of 7 (width 7168 in heads of 128) and 3, and one query head to each head of the cache.
HEADS = ((32, 4, 128), (16, 2, 256), (56, 8, 128), (24, 8, 64), (8, 8, 128))
TYPES = ("bf16", "mxfp8", "mxfp4")
LIMIT = {"mxfp8": (448.0, 7), "mxfp4": (6.0, 13)}


def _case(op, kind, heads, page, **more):
    return {"op": op, "type": kind, "heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "page": page, **more}


def listed():
    a, b, c, d, e = HEADS
    return [
        # one token's rows in a batch-1 decode step: latency
        {"name": "write 1 token mxfp8", **_case("write", "mxfp8", a, 16, tokens=1, skip=0)},
        # a prefill chunk of 8192 tokens
        {"name": "write 8192 tokens mxfp4", **_case("write", "mxfp4", b, 64, tokens=8192, skip=0)},
        # a padded mixed batch: every 16th row is padding and goes nowhere
        {"name": "write 777 padded bf16", **_case("write", "bf16", d, 32, tokens=777, skip=16)},
        # a short prefix, and a long session's whole cache, as dense rows
        {"name": "read 300 tokens mxfp4", **_case("read", "mxfp4", c, 16, tokens=300, skip=0)},
        {"name": "read 131072 tokens mxfp8", **_case("read", "mxfp8", a, 64, tokens=131072, skip=0)},
        # decode: one session, then a full batch of sessions of very different lengths
        {"name": "attn decode 1x4001 bf16", **_case("attn", "bf16", b, 16, seqs=1, new=1, new_min=1, kv=4001, kv_min=4001, window=0)},
        {"name": "attn decode 64x<=32768 mxfp8", **_case("attn", "mxfp8", a, 64, seqs=64, new=1, new_min=1, kv=32768, kv_min=1, window=0)},
        # four drafted tokens of each of 16 sessions checked at once, in groups of 7 heads
        {"name": "attn verify 16x4 mxfp4", **_case("attn", "mxfp4", c, 32, seqs=16, new=4, new_min=4, kv=16411, kv_min=1000, window=0)},
        # a prompt's first chunk, the whole of it new
        {"name": "attn chunk 8192 bf16", **_case("attn", "bf16", a, 64, seqs=1, new=8192, new_min=8192, kv=8192, kv_min=8192, window=0)},
        # a later chunk of a long prompt
        {"name": "attn chunk 2048 over 65536 mxfp8", **_case("attn", "mxfp8", a, 64, seqs=1, new=2048, new_min=2048, kv=65536, kv_min=65536, window=0)},
        # a few new tokens of a very long session, with wide heads
        {"name": "attn chunk 500 over 100001 bf16", **_case("attn", "bf16", b, 128, seqs=1, new=500, new_min=500, kv=100001, kv_min=100001, window=0)},
        # chunks and single tokens in one batch, with a sliding window
        {"name": "attn mixed 12x<=1025 window", **_case("attn", "bf16", d, 16, seqs=12, new=1025, new_min=1, kv=9000, kv_min=1025, window=1024)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv, page = rng.choice(HEADS), rng.choice(TYPES), rng.choice((16, 32, 64, 128))
    op = rng.choice(("write", "read", "attn", "attn", "attn"))
    if op == "write":
        return _case(op, kv, heads, page, tokens=_log(rng, 1, 8192), skip=rng.choice((0, 0, 7, 16)))
    if op == "read":
        return _case(op, kv, heads, page, tokens=_log(rng, 100, 65536), skip=rng.choice((0, 0, 9)))
    form = rng.choice(("decode", "verify", "chunk", "mixed"))
    window = rng.choice((0, 0, rng.randint(100, 4096)))
    if form in ("decode", "verify"):
        new = 1 if form == "decode" else rng.randint(2, 16)
        kv_max = _log(rng, 64, 65536)
        seqs = _log(rng, 1, max(1, min(64, 2_000_000 // (kv_max * new))))
        return _case("attn", kv, heads, page, seqs=seqs, new=new, new_min=new, kv=kv_max, kv_min=rng.randint(new, kv_max), window=window)
    if form == "chunk":
        new = _log(rng, 33, 8192)
        kv_max = min(131072, max(new, _log(rng, new, max(new, 67_000_000 // new))))
        if 4 * heads[0] * heads[2] * new * kv_max > 2.0e12:  # stay below the largest listed case
            kv_max = max(new, int(2.0e12 / (4 * heads[0] * heads[2] * new)))
        return _case("attn", kv, heads, page, seqs=1, new=new, new_min=new, kv=kv_max, kv_min=kv_max, window=window)
    seqs, new = rng.randint(2, 16), _log(rng, 16, 1025)
    return _case("attn", kv, heads, page, seqs=seqs, new=new, new_min=1, kv=new + _log(rng, 100, 8000), kv_min=new, window=window)


def _spread(lo, hi, n):
    """n lengths from lo to hi, in even steps of their logarithm, short and long ones in turn."""
    v = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) if lo < hi else hi for i in range(n)]
    v[-1] = hi
    return v[0::2] + v[1::2][::-1]


def _lengths(c):
    """(new, cached) tokens of every sequence: the cached ones include the new ones."""
    new = _spread(c["new_min"], c["new"], c["seqs"])
    kv = _spread(c["kv_min"], c["kv"], c["seqs"])[::-1]
    return new, [max(a, b) for a, b in zip(new, kv)]


def _row_bytes(c):
    """Bytes of one row of one head: elements and scales."""
    return c["dim"] * 2 if c["type"] == "bf16" else c["dim"] // (1 if c["type"] == "mxfp8" else 2) + c["dim"] // 32


def work(case):
    c = case
    row = 2 * c["kv_heads"] * _row_bytes(c)   # a token's keys and values, as cached
    dense = 2 * c["kv_heads"] * c["dim"] * 2  # the same in BF16
    if c["op"] != "attn":
        n, skipped = c["tokens"], -(-c["tokens"] // c["skip"]) if c["skip"] else 0
        return {"bytes": n * 4 + (n - skipped) * row + n * dense + ((n - skipped) * dense if c["op"] == "write" else 0),
                "flops": 2 * (n - skipped) * c["kv_heads"] * c["dim"]}
    pairs = rows = total = 0
    for n, kv in zip(*_lengths(c)):
        first, w = kv - n, c["window"] or kv
        full = max(0, n - max(0, w - first - 1))  # rows whose window is full
        part = n - full
        pairs += full * w + part * (first + 1) + part * (part - 1) // 2
        rows += kv - max(0, first + 1 - w)
        total += n
    q = total * c["heads"] * c["dim"] * 2
    return {"bytes": 2 * q + total * c["heads"] * 4 + rows * row, "flops": 4 * pairs * c["heads"] * c["dim"]}


# ------------------------------------------------------------------ plain forms


def _quantise(x, kv):
    """FP32 rows [..., dim] -> (element codes as bytes, scale codes)."""
    top, cap = LIMIT[kv]
    b = x.unflatten(-1, (-1, 32))
    m, ex = torch.frexp(b.abs().amax(-1))
    mt, et = math.frexp(top)
    e = torch.where(m > mt, ex - et + 1, ex - et).clamp(-100, cap)
    y = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-top, top)
    if kv == "mxfp8":
        code = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:
        a = y.abs()
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
                + torch.signbit(y) * 8).to(torch.uint8).flatten(-2)
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, (e + 127).to(torch.uint8)


def _stands_for(code, scale, kv):
    """The FP32 values that element codes and scales stand for."""
    if kv == "bf16":
        return code.float()
    if kv == "mxfp8":
        v = code.view(torch.float8_e4m3fn).float()
    else:
        code = torch.stack((code & 15, code >> 4), -1).flatten(-2)
        ee, m = ((code >> 1) & 3).int(), (code & 1).float()
        v = torch.where(ee > 0, torch.ldexp(1 + m / 2, ee - 1), m / 2)
        v = torch.where(code > 7, -v, v)
    return torch.ldexp(v.unflatten(-1, (-1, 32)), (scale.int() - 127).unsqueeze(-1)).flatten(-2)


def _take(s, slots):
    """Rows of the given slots (-1: zeros) as BF16: [n, kv_heads, dim] of keys and of values."""
    page, off = torch.where(slots < 0, s["spare"], slots // s["page"]).long(), (slots % s["page"]).long()
    got = []
    for name in ("k", "v"):
        scale = s[name + "_scale"]
        x = _stands_for(s[name][page, :, off], None if scale is None else scale[page, :, off], s["type"])
        got.append(torch.where((slots >= 0)[:, None, None], x, 0.0).to(torch.bfloat16))
    return got


def _put(s, slots):
    page, off = torch.where(slots < 0, s["spare"], slots // s["page"]).long(), (slots % s["page"]).long()
    for name in ("k", "v"):
        x = s["new_" + name]
        if s["type"] == "bf16":
            s[name][page, :, off] = x
        else:
            code, scale = _quantise(x.float(), s["type"])
            s[name][page, :, off] = code
            s[name + "_scale"][page, :, off] = scale


def _attend(s):
    """Every sequence padded to the longest."""
    heads, kvh, dim, new = s["heads"], s["kv_heads"], s["dim"], s["new"]
    start, length, table = s["q_start"].long(), s["kv_len"].long(), s["table"].long()
    n = start[1:] - start[:-1]
    at = torch.arange(new, device="cuda")
    q = s["q"][(start[:-1, None] + at).clamp(max=s["q"].shape[0] - 1)].float()  # [seqs, new, heads, dim]
    q = q.unflatten(2, (kvh, -1)).permute(0, 2, 3, 1, 4)                        # [seqs, kv_heads, group, new, dim]
    rows = []
    for name in ("k", "v"):
        scale = s[name + "_scale"]
        x = _stands_for(s[name][table], None if scale is None else scale[table], s["type"])
        rows.append(x.permute(0, 2, 1, 3, 4).flatten(2, 3))                     # [seqs, kv_heads, cached, dim]
    k, v = rows
    z = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (-1, new)).mul_(s["scale"])
    p = (length - n)[:, None] + at                                              # position of each new token
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j <= p[..., None]) & (j < length[:, None, None])
    if s["window"]:
        seen &= j > p[..., None] - s["window"]
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    out = torch.matmul(z.flatten(2, 3), v).unflatten(2, (-1, new)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]
    seq, i = s["seq_of"], s["place"]
    out = out.permute(0, 3, 1, 2, 4)[seq, i].flatten(1, 2).to(torch.bfloat16)   # [tokens, heads, dim]
    return out, lse.permute(0, 3, 1, 2)[seq, i].flatten(1, 2)


# ------------------------------------------------------------------ one pass


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kvh, dim, page, kv = c["kv_heads"], c["dim"], c["page"], c["type"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # some channels of the keys are far larger than the others, as trained models have them
    gain = torch.exp(0.5 * normal(kvh, 1, dim))
    s = {**c, "spare": torch.zeros((), dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(dim)}
    if c["op"] == "attn":
        new, length = _lengths(c)
        pages = [-(-n // page) for n in length]
        wide = max(pages)
    else:
        pages, wide = [c["tokens"] // page + 2], 0
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages - 1, generator=g, device="cuda").int() + 1  # page 0 belongs to nobody
    for name in ("k", "v"):
        if c["op"] == "write":  # the cache before its first tokens
            x = torch.zeros(n_pages, kvh, page, dim, device="cuda")
        else:
            x = normal(n_pages, kvh, page, dim)
            if name == "k":
                x *= gain
        s[name], s[name + "_scale"] = (x.to(torch.bfloat16), None) if kv == "bf16" else _quantise(x, kv)
        del x
    if c["op"] == "attn":
        t = torch.zeros(c["seqs"], wide, dtype=torch.int32)
        at, host = 0, order.cpu()
        for i, n in enumerate(pages):
            t[i, :n] = host[at:at + n]
            at += n
        start = torch.tensor([0] + new).cumsum(0)
        total = int(start[-1])
        s["table"], s["q_start"] = t.cuda(), start.int().cuda()
        s["kv_len"] = torch.tensor(length, dtype=torch.int32).cuda()
        s["seq_of"] = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(new)).cuda()
        s["place"] = torch.arange(total).cuda() - s["q_start"].long()[s["seq_of"]]
        s["q"] = normal(total, c["heads"], dim).to(torch.bfloat16)
    else:
        n, first = c["tokens"], seed % page  # tokens begin inside a page
        at = torch.arange(n, device="cuda", dtype=torch.int32) + first
        slots = order[(at // page).long()] * page + at % page
        if c["skip"]:
            slots[:: c["skip"]] = -1
        s["slots"] = slots
        if c["op"] == "write":  # keys and values are parts of one projection's rows, the queries before them
            qkv = normal(n, c["heads"] + 2 * kvh, dim)
            qkv[:, c["heads"]:c["heads"] + kvh] *= gain[:, 0]
            s["qkv"] = qkv.to(torch.bfloat16)
            s["new_k"], s["new_v"] = s["qkv"][:, c["heads"]:c["heads"] + kvh], s["qkv"][:, c["heads"] + kvh:]
    if own:
        from serving_router_top_dedupe_gb300 import ftmoe as F

        kind = {"bf16": F.FT_KV_BF16, "mxfp8": F.FT_KV_MXFP8, "mxfp4": F.FT_KV_MXFP4}[kv]
        s["cache"] = F.make_kv_cache(kind, kvh, dim, page, n_pages, s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] == "attn":
            s["workspace"] = torch.zeros(F.ft_attn_workspace(c["heads"], kvh, dim), dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
            s["args"] = F.make_attn_args(c["heads"], c["new"], s["q"], s["q_start"], s["kv_len"], s["table"], s["out"],
                                         s["workspace"], scale=s["scale"], window=c["window"], lse=s["lse"])
        else:
            s["k_out"], s["v_out"] = (torch.empty(c["tokens"], kvh, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    return s


def run(state):
    s = state
    if not own:
        if s["op"] == "attn":
            return _attend(s)
        if s["op"] == "write":
            _put(s, s["slots"])
        return _take(s, s["slots"])
    from serving_router_top_dedupe_gb300 import ftmoe as F

    stream = torch.cuda.current_stream().cuda_stream
    if s["op"] == "attn":
        F.ft_attn(s["cache"], s["args"], stream=stream)
        return s["out"], s["lse"]
    if s["op"] == "write":
        F.ft_kv_write(s["cache"], s["new_k"], s["new_v"], s["slots"], stream=stream)
    F.ft_kv_read(s["cache"], s["slots"], s["k_out"], s["v_out"], stream=stream)
    return [s["k_out"], s["v_out"]]


# ------------------------------------------------------------------ the definition in 64 bits


def _rounded(x, kv):
    """What a row of 64-bit values reads back as."""
    top, cap = LIMIT[kv]
    b = x.reshape(*x.shape[:-1], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0) / top))
    e = torch.where(a > top * torch.exp2(e), e + 1, e)  # the smallest e with a <= top * 2^e
    e = torch.where(a <= top * torch.exp2(e - 1), e - 1, e)
    e = torch.where(a > 0, e, -100.0).clamp(-100, cap)
    y = (b * torch.exp2(-e)).clamp(-top, top)
    low, bits = (-6, 3) if kv == "mxfp8" else (0, 1)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))) - bits)
    return (torch.round(y / step) * step * torch.exp2(e)).reshape(x.shape)


def _values64(code, scale, kv):
    """64-bit values of cached rows, from the bits of the formats."""
    if kv == "bf16":
        return code.double()
    if kv == "mxfp4":
        code = torch.stack((code % 16, code // 16), -1).reshape(*code.shape[:-1], -1)
    bias, bits, sign = (7, 3, 128) if kv == "mxfp8" else (1, 1, 8)
    every = torch.arange(256 if kv == "mxfp8" else 16, dtype=torch.float64)
    mag = every % sign
    ex, frac = torch.floor(mag / 2 ** bits), (mag % 2 ** bits) / 2 ** bits
    value = torch.where(ex > 0, (1 + frac) * torch.exp2(ex - bias), frac * 2.0 ** (1 - bias))
    value = torch.where(every >= sign, -value, value).to(code.device)
    x = value[code.long()]
    return x * torch.exp2(scale.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    kv, page = s["type"], s["page"]
    if s["op"] != "attn":
        slots = s["slots"]
        keep = (slots >= 0)[:, None, None].double()
        p, o = (slots.clamp(min=0) // page).long(), (slots.clamp(min=0) % page).long()
        got = []
        for name in ("k", "v"):
            if s["op"] == "write":
                x = s["new_" + name].double()
                x = x if kv == "bf16" else _rounded(x, kv)
            else:
                x = _values64(s[name][p, :, o], None if kv == "bf16" else s[name + "_scale"][p, :, o], kv)
            got.append(x * keep)
        return got
    heads, kvh = s["heads"], s["kv_heads"]
    new, length = _lengths(s)
    outs, lses = [], []
    at = 0
    for i, (n, kl) in enumerate(zip(new, length)):
        pages = s["table"][i, : -(-kl // page)].long()
        out = torch.empty(n, heads, s["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(n, heads, dtype=torch.float64, device="cuda")
        for h in range(kvh):
            k, v = (_values64(s[x][pages, h].reshape(len(pages) * page, -1),
                              None if kv == "bf16" else s[x + "_scale"][pages, h].reshape(len(pages) * page, -1), kv)
                    for x in ("k", "v"))
            for r in range(0, n, 1024):
                m = min(1024, n - r)
                pos = kl - n + r + torch.arange(m, device="cuda")
                hi = kl - n + r + m
                lo = max(0, kl - n + r - s["window"] + 1) if s["window"] else 0
                j = torch.arange(lo, hi, device="cuda")
                hide = j[None] > pos[:, None]
                if s["window"]:
                    hide = hide | (j[None] + s["window"] <= pos[:, None])
                group = slice(h * heads // kvh, (h + 1) * heads // kvh)
                q = s["q"][at + r:at + r + m, group].double().transpose(0, 1)  # [group, m, dim]
                z = torch.matmul(q, k[lo:hi].T) * s["scale"]
                z.masked_fill_(hide, -math.inf)
                norm = torch.logsumexp(z, -1)
                out[r:r + m, group] = torch.matmul(torch.exp(z - norm[..., None]), v[lo:hi]).transpose(0, 1)
                lse[r:r + m, group] = norm.T
        outs.append(out)
        lses.append(lse)
        at += n
    return torch.cat(outs), torch.cat(lses)
