"""The example's calls follow one another: a model run as it is gives the same bits as one that waits for the GPU before and after
every call of the MoE half."""
import pytest
import torch

from test_gpu_example import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def _run(E, cache):
    m = E.Layers(cache, max_tokens=150, chunk=48)
    try:
        g = torch.Generator(device="cuda")
        g.manual_seed(11)
        x = m.prompt(torch.randn(120, m.w.hidden, generator=g, device="cuda").to(torch.bfloat16))
        states = [x]
        for _ in range(12):
            x = m.forward(E.norm(x))
            states.append(x)
        torch.cuda.synchronize()
        assert m.error.item() == 0 and E.F.ft_moe_get_stats(m.moe).error_word == 0
        return torch.cat(states).cpu()
    finally:
        m.close()


def test_the_moe_half_is_on_a_stream_that_was_named(example):  # noqa: F811
    m = example.Layers("bf16", max_tokens=16, chunk=8)
    try:
        assert m.stream
    finally:
        m.close()


@pytest.mark.parametrize("cache", ["bf16", "mxfp8", "mxfp4"])
def test_states_do_not_depend_on_when_calls_run(example, cache, monkeypatch):  # noqa: F811
    E = example
    first = _run(E, cache)
    for name in ("ft_moe_decode_step_hidden", "ft_moe_prefill_chunk_hidden"):
        def waits(*a, _call=getattr(E.F, name), **k):
            torch.cuda.synchronize()
            _call(*a, **k)
            torch.cuda.synchronize()

        monkeypatch.setattr(E.F, name, waits)
    want = _run(E, cache)
    assert torch.isfinite(want).all()
    monkeypatch.undo()
    for got in (first, _run(E, cache), _run(E, cache)):
        assert torch.equal(got, want)
