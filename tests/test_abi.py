"""C-ABI checks that need no GPU: the library loads, exports every entry point the
header declares, the host split mirror agrees with the oracle, and argument
errors come back as status codes."""
import os
import random
import re

import numpy as np
import pytest

import oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def F():
    import __graft_entry__ as g

    g.build()
    from serving_router_top_dedupe_gb300 import ftmoe

    return ftmoe


def _declared():
    names = set()
    for fn in os.listdir(os.path.join(ROOT, "include")):
        text = open(os.path.join(ROOT, "include", fn)).read()
        names |= set(re.findall(r"^\s*(?:ft_status|const char\*)\s+(ft_\w+)\s*\(", text, re.M))
    return names


def test_library_exports_every_declared_symbol(F):
    declared = _declared()
    assert len(declared) >= 20
    import ctypes

    lib = ctypes.CDLL(F.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    assert declared == set(F.EXPORTED)


def test_binding_argument_counts_match_the_header(F):
    """Every declared entry point takes as many arguments in the binding's ctypes
    signature as in the C declaration."""
    arity = {}
    for fn in os.listdir(os.path.join(ROOT, "include")):
        text = open(os.path.join(ROOT, "include", fn)).read()
        for m in re.finditer(r"^\s*(?:ft_status|const char\*)\s+(ft_\w+)\s*\(([^)]*)\)\s*;", text, re.M):
            args = m.group(2).strip()
            arity[m.group(1)] = 0 if args in ("", "void") else args.count(",") + 1
    assert len(arity) >= 20
    for name, n in arity.items():
        if name in F._SIGS:
            assert len(F._SIGS[name]) == n, name


def test_split_host_mirror_matches_oracle(F):
    rng = random.Random(3)
    for _ in range(2000):
        m = rng.randint(0, 300)
        bp = round(rng.uniform(0.5, 400), 3)
        bh = round(rng.uniform(0.5, 400), 3)
        ev = rng.randint(0, 400)
        assert F.ft_split_misses(m, bp, bh, ev) == O.split_misses(m, O.mbps(bp), O.mbps(bh), ev)
    assert F.ft_split_misses(4, 11.8, 47.5, 99) == 1
    assert F.ft_split_misses(4, 52.7, 77.3, 99) == 3


def test_split_rejects_bad_arguments(F):
    for args in [(-1, 1.0, 1.0, 1), (1, 0.0, 1.0, 1), (1, 1.0, -2.0, 1), (1, 1.0, 1.0, -1)]:
        with pytest.raises(F.FtError) as e:
            F.ft_split_misses(*args)
        assert e.value.status == F.FT_ERR_INVALID


def test_init_rejects_bad_config_without_touching_the_gpu(F):
    banks = {"gate": np.zeros(16, np.uint16), "up": np.zeros(16, np.uint16), "down": np.zeros(16, np.uint16)}
    bad = [
        dict(hidden=100),           # not a multiple of 256
        dict(top_k=0), dict(top_k=17), dict(n_experts=2000), dict(max_batch=65), dict(cache_slots=0),
        dict(inter=100), dict(bh_gbps=0.0), dict(wtype=7),
    ]
    base = dict(n_layers=2, hidden=256, inter=128, n_experts=16, top_k=2, has_shared=False, wtype=F.FT_W_BF16,
                max_batch=1, cache_slots=8, bp_gbps=11.8, bh_gbps=47.5)
    for b in bad:
        with pytest.raises(F.FtError) as e:
            F.ft_moe_init(F.make_config(**{**base, **b}), banks)
        assert e.value.status == F.FT_ERR_INVALID
    with pytest.raises(F.FtError) as e:  # FP8 without scale banks
        F.ft_moe_init(F.make_config(**{**base, "wtype": F.FT_W_FP8_E4M3_B128, "hidden": 512}), banks)
    assert e.value.status == F.FT_ERR_INVALID
    u8 = np.zeros(16, np.uint8)
    for wt in (F.FT_W_NVFP4, F.FT_W_MXFP4):  # block-FP4 without their scale banks
        with pytest.raises(F.FtError) as e:
            F.ft_moe_init(F.make_config(**{**base, "wtype": wt}), {"gate": u8, "up": u8, "down": u8})
        assert e.value.status == F.FT_ERR_INVALID
    with pytest.raises(F.FtError) as e:  # NVFP4 needs the tensor scales too
        F.ft_moe_init(F.make_config(**{**base, "wtype": F.FT_W_NVFP4}),
                      {"gate": u8, "up": u8, "down": u8, "gate_bscale": u8, "up_bscale": u8, "down_bscale": u8})
    assert e.value.status == F.FT_ERR_INVALID


def test_router_and_prefill_calls_reject_a_null_handle(F):
    for call in (lambda: F.ft_moe_set_router(None, None, 0), lambda: F.ft_moe_router_logits(None, 0, 1, 1, 1),
                 lambda: F.ft_moe_decode_step_hidden(None, 0, 1, 1, 1, 1),
                 lambda: F.ft_moe_prefill_chunk_hidden(None, 0, 1, 1, 1),
                 lambda: F.ft_moe_prefill_chunk(None, 0, 1, 1, 1, 1),
                 lambda: F.ft_moe_set_host_hook(None, None), lambda: F.ft_moe_set_prefill_overlap(None, True)):
        with pytest.raises(F.FtError) as e:
            call()
        assert e.value.status == F.FT_ERR_INVALID


def test_null_handle_calls_fail_cleanly(F):
    with pytest.raises(F.FtError):
        F.ft_moe_decode_step(None, 0, 1, 1, 1, 1, 1)
    with pytest.raises(F.FtError):
        F.ft_cache_resize(None, 4)
    with pytest.raises(F.FtError):
        F.ft_moe_get_stats(None)
    F.ft_moe_destroy(None)


def test_binding_without_the_library_fails_loudly(tmp_path):
    """The binding has no fallback: a copy of the package without the built library
    raises at import."""
    import shutil
    import subprocess
    import sys

    pkg = tmp_path / "serving_router_top_dedupe_gb300"
    pkg.mkdir()
    for fn in ("__init__.py", "ftmoe.py"):
        shutil.copy(os.path.join(ROOT, "serving_router_top_dedupe_gb300", fn), pkg / fn)
    r = subprocess.run([sys.executable, "-c", "import serving_router_top_dedupe_gb300.ftmoe"], cwd=tmp_path,
                       capture_output=True, text=True, timeout=120,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode != 0
    assert "ImportError" in r.stderr and "libftmoe.so is missing" in r.stderr


def _kv(F, **change):
    a = dict(kv_type=F.FT_KV_MXFP8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=4, k=4096, v=8192, k_scale=256, v_scale=512)
    a.update(change)
    return F.ft_kv_cache(*a.values())


def _attn(F, **change):
    a = dict(n_heads=4, n_tokens=3, n_seqs=2, max_new=2, table_stride=4, causal=1, window=0, scale=0.1, q=4096, q_stride=512,
             q_start=4, kv_len=4, page_table=4, out=4096, out_stride=512, lse=0, workspace=256, workspace_bytes=1 << 40,
             error_word_out=0)
    a.update(change)
    return F.ft_attn_args(*a.values())


def test_cache_calls_reject_bad_arguments_without_touching_the_gpu(F):
    import ctypes as C

    def bad(st):
        assert st == F.FT_ERR_INVALID and F.ft_last_error()

    caches = [None, dict(kv_type=3), dict(n_kv_heads=0), dict(n_kv_heads=2000), dict(head_dim=96), dict(page_size=8),
              dict(page_size=48), dict(n_pages=0), dict(n_pages=1 << 30), dict(k=None), dict(v_scale=None), dict(k=4100),
              dict(k_scale=8)]
    for ch in caches:
        c = None if ch is None else C.byref(_kv(F, **ch))
        bad(F._lib.ft_kv_write(c, 1, 4096, 4096, 256, 256, 4, None, None))
        bad(F._lib.ft_kv_read(c, 1, 4, 4096, 4096, 256, 256, None, None))
        bad(F._lib.ft_attn(c, C.byref(_attn(F)), None))
    c = C.byref(_kv(F))
    for args in [(-1, 4096, 4096, 256, 256, 4), (1, None, 4096, 256, 256, 4), (1, 4096, 4098, 256, 256, 4),
                 (1, 4096, 4096, 252, 256, 4), (1, 4096, 4096, 256, -256, 4), (1, 4096, 4096, 256, 256, None)]:
        bad(F._lib.ft_kv_write(c, *args, None, None))
        bad(F._lib.ft_kv_read(c, args[0], args[5], *args[1:5], None, None))
    bad(F._lib.ft_kv_read(c, 2, 4, 4096, 4096, 248, 256, None, None))  # rows that overlap
    for ch in [dict(n_heads=3), dict(n_heads=0), dict(n_heads=2 * 129), dict(n_tokens=-1), dict(n_seqs=1025), dict(n_seqs=-1),
               dict(max_new=0), dict(table_stride=0), dict(table_stride=1 << 28), dict(causal=2), dict(window=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=4104), dict(out=None), dict(q_stride=12),
               dict(out_stride=256), dict(q_start=None), dict(kv_len=None), dict(page_table=2), dict(workspace=None),
               dict(workspace=128), dict(lse=2), dict(n_tokens=1 << 30)]:
        bad(F._lib.ft_attn(c, C.byref(_attn(F, **ch)), None))
    bad(F._lib.ft_attn(c, None, None))
    n = C.c_size_t()
    for args in [(3, 2, 128), (0, 1, 128), (4, 0, 128), (4, 2, 100), (300, 2, 64)]:
        bad(F._lib.ft_attn_workspace(*args, C.byref(n)))
    bad(F._lib.ft_attn_workspace(4, 2, 128, None))


def test_cache_calls_without_tokens_do_nothing(F):
    import ctypes as C

    c = C.byref(_kv(F))
    assert F._lib.ft_kv_write(c, 0, None, None, 0, 0, None, None, None) == F.FT_OK
    assert F._lib.ft_kv_read(c, 0, None, None, None, 0, 0, None, None) == F.FT_OK
    assert F._lib.ft_attn(c, C.byref(_attn(F, n_tokens=0, q=None)), None) == F.FT_OK
    assert F._lib.ft_attn(c, C.byref(_attn(F, n_seqs=0)), None) == F.FT_OK


def test_cache_binding_checks_its_tensors(F):
    import torch

    k = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 16, 4, dtype=torch.uint8)
    c = F.make_kv_cache(F.FT_KV_MXFP8, 2, 128, 16, 4, k, k, sc, sc)
    for args in [(F.FT_KV_MXFP8, 2, 128, 16, 5, k, k, sc, sc), (F.FT_KV_BF16, 2, 128, 16, 4, k, k),
                 (F.FT_KV_MXFP8, 2, 128, 16, 4, k, k, None, sc), (F.FT_KV_MXFP4, 2, 128, 16, 4, k, k, sc, sc), (9, 2, 128, 16, 4, k, k),
                 (F.FT_KV_MXFP8, 2, 128, 16, 4, k.transpose(0, 1), k, sc, sc)]:
        with pytest.raises(ValueError):
            F.make_kv_cache(*args)
    x, slots = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for kk, v, s in [(x.float(), x, slots), (x, x[:2], slots), (x, x, slots.long()), (x, x, slots[:2]), (x[:, :1], x, slots),
                     (x.transpose(1, 2), x, slots), (torch.zeros(3, 2, 256, dtype=torch.bfloat16)[..., ::2], x, slots)]:
        with pytest.raises(ValueError):
            F.ft_kv_write(c, kk, v, s)
        with pytest.raises(ValueError):
            F.ft_kv_read(c, s, kk, v)
    q, i32 = torch.zeros(3, 4, 128, dtype=torch.bfloat16), lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    ok = dict(q=q, q_start=i32(3), kv_len=i32(2), page_table=i32(2, 4), out=q, workspace=ws, lse=torch.zeros(3, 4))
    F.make_attn_args(4, 1, **ok, scale=1.0)
    for ch in [dict(q=q.float()), dict(q=q[:2]), dict(out=q[:, :2]), dict(q_start=i32(2)), dict(page_table=i32(3, 4)),
               dict(kv_len=torch.zeros(2, dtype=torch.int64)), dict(lse=torch.zeros(3, 3))]:
        with pytest.raises(ValueError):
            F.make_attn_args(4, 1, **{**ok, **ch}, scale=1.0)
    other = F.make_attn_args(4, 1, **{**ok, "q": q[..., :64].contiguous(), "out": q[..., :64].contiguous()}, scale=1.0)
    with pytest.raises(ValueError):
        F.ft_attn(c, other)
