"""What the binding of the paged cache refuses before it hands addresses to the library: other types of the same size, tensors
that the GPU cannot read, workspaces with gaps.  No GPU is needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def F():
    from serving_router_top_dedupe_gb300 import ftmoe

    return ftmoe


class Seen(torch.Tensor):
    """A tensor that says that it is on the GPU."""

    is_cuda = True


def _cache(F, on_gpu=True, kind=1):
    like = (lambda t: t.as_subclass(Seen)) if on_gpu else (lambda t: t)
    k, v = (like(torch.zeros(4, 2, 16, 128, dtype=torch.uint8 if kind else torch.bfloat16)) for _ in "kv")
    ks, vs = (like(torch.zeros(4, 2, 16, 4, dtype=torch.uint8)) for _ in "kv")
    return F.make_kv_cache(kind, 2, 128, 16, 4, k, v, ks, vs)


def _args(F, **change):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    a = dict(q=q, q_start=i32(3), kv_len=i32(2), page_table=i32(2, 4), out=q, workspace=torch.zeros(64, dtype=torch.uint8),
             lse=torch.zeros(3, 4), error_word=i32(1))
    a.update(change)
    return F.make_attn_args(4, 1, **a, scale=1.0)


def test_other_types_of_the_same_size_are_refused(F):
    half, f32, i32 = (torch.zeros(3, 4, 128).half(), torch.zeros(3, 4), lambda *s: torch.zeros(*s, dtype=torch.int32))
    _args(F)
    _args(F, q=torch.zeros(3, 4, 128, dtype=torch.int16), error_word=None, lse=None)  # BF16 patterns are fine
    for change in (dict(q=half), dict(out=half), dict(q_start=f32[0, :3]), dict(kv_len=torch.zeros(2)), dict(page_table=torch.zeros(2, 4)),
                   dict(lse=i32(3, 4)), dict(error_word=torch.zeros(1)), dict(error_word=i32(0)), dict(error_word=i32(1).long()),
                   dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])):
        with pytest.raises(ValueError):
            _args(F, **change)
    k = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 16, 4, dtype=torch.uint8)
    for bad in (dict(k=k.bool()), dict(k_scale=sc.bool())):
        with pytest.raises(ValueError):
            F.make_kv_cache(F.FT_KV_MXFP8, 2, 128, 16, 4, **{**dict(k=k, v=k, k_scale=sc, v_scale=sc), **bad})
    with pytest.raises(ValueError):
        F.make_kv_cache(F.FT_KV_BF16, 2, 128, 16, 4, *(torch.zeros(4, 2, 16, 128).half() for _ in "kv"))
    F.make_kv_cache(F.FT_KV_MXFP8, 2, 128, 16, 4, k.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), sc, sc)


def test_rows_of_other_types_are_refused(F, monkeypatch):
    monkeypatch.setattr(F, "_lib", None)  # nothing may be called
    c = _cache(F)
    seen = lambda *s, dtype: torch.zeros(*s, dtype=dtype).as_subclass(Seen)
    x, slots = seen(3, 2, 128, dtype=torch.bfloat16), seen(3, dtype=torch.int32)
    for k, v, s, word in [(seen(3, 2, 128, dtype=torch.float16), x, slots, None), (x, seen(3, 2, 128, dtype=torch.float16), slots, None),
                          (x, x, seen(3, dtype=torch.float32), None), (x, x, slots, seen(1, dtype=torch.float32))]:
        with pytest.raises(ValueError):
            F.ft_kv_write(c, k, v, s, error_word=word)
        with pytest.raises(ValueError):
            F.ft_kv_read(c, s, k, v, error_word=word)


def test_tensors_that_are_not_on_the_gpu_are_refused(F, monkeypatch):
    monkeypatch.setattr(F, "_lib", None)
    seen = lambda *s, dtype: torch.zeros(*s, dtype=dtype).as_subclass(Seen)
    x, slots = seen(3, 2, 128, dtype=torch.bfloat16), seen(3, dtype=torch.int32)
    host = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    word = torch.zeros(1, dtype=torch.int32)
    for cache, k, v, s, w in [(_cache(F, False), x, x, slots, None), (_cache(F), host, x, slots, None), (_cache(F), x, host, slots, None),
                              (_cache(F), x, x, torch.zeros(3, dtype=torch.int32), None), (_cache(F), x, x, slots, word)]:
        with pytest.raises(ValueError, match="GPU"):
            F.ft_kv_write(cache, k, v, s, error_word=w)
        with pytest.raises(ValueError, match="GPU"):
            F.ft_kv_read(cache, s, k, v, error_word=w)
    with pytest.raises(ValueError, match="GPU"):
        F.ft_attn(_cache(F), _args(F))
    on = {n: seen(*s, dtype=d) for n, s, d in [("q", (3, 4, 128), torch.bfloat16), ("out", (3, 4, 128), torch.bfloat16),
                                               ("q_start", (3,), torch.int32), ("kv_len", (2,), torch.int32), ("lse", (3, 4), torch.float32),
                                               ("page_table", (2, 4), torch.int32), ("workspace", (64,), torch.uint8), ("error_word", (1,), torch.int32)]}
    with pytest.raises(ValueError, match="GPU"):
        F.ft_attn(_cache(F, False), _args(F, **on))
    for name, t in on.items():
        with pytest.raises(ValueError, match="GPU"):
            F.ft_attn(_cache(F), _args(F, **{**on, name: t.as_subclass(torch.Tensor)}))
    with pytest.raises(AttributeError):  # all there: the library (taken away here) is what comes next
        F.ft_attn(_cache(F), _args(F, **on))


def test_the_constants_are_those_of_the_header(F):
    import os
    import re

    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ft_kv.h")) as f:
        text = f.read().replace("(size_t)", "")
    for name in ("FT_ATTN_CLEAR_BYTES", "FT_ATTN_COPY_BYTES"):
        assert eval(re.search(rf"#define {name} (.*)", text)[1]) == getattr(F, name)
