"""CPU tests of AttentionBuffers.run's refusals: a layer, cache or batch that
does not fit the buffers is refused before any entry point that launches work
has been called."""

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R

LAUNCHES = ("quantize_act", "gemv_grouped", "gemm", "qk_norm_rope", "attn")


def layer(hidden=64, heads=4, kv_heads=2, dim=16, fmt=4, **kw):
    return R.DeviceAttention.build(hidden, heads, kv_heads, dim, lambda m, r, c: np.ones((r, c), np.float32), fmt=fmt,
                                   device="cpu", **kw)


def cache(kv_heads=2, dim=16, page=16, dtype=torch.float16):
    return R.DeviceKVCache(*(torch.zeros(4, kv_heads, page, dim, dtype=dtype) for _ in range(2)))


def batch(tokens, max_q=None, seqs=1, width=4):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return R.KVBatch(i(seqs + 1), i(seqs), i(seqs, width), tokens, max_q or tokens)


@pytest.fixture
def launched(monkeypatch):
    calls = []
    for name in LAUNCHES:
        monkeypatch.setattr(R, name, lambda *a, _n=name, **k: calls.append(_n))
    return calls


@pytest.mark.parametrize("T", [1, 3, 6, 40])
def test_what_does_not_fit_is_refused_before_any_launch(T, launched):
    own, c, b = layer(), cache(), batch(T)
    buf = R.AttentionBuffers(own, c, b, device="cpu")
    x = torch.zeros(T, 64)
    wide = torch.zeros(T, 96)
    cases = {
        "more kv heads": (layer(kv_heads=4), x, cache(kv_heads=4), b, {}),
        "fewer kv heads": (layer(kv_heads=1), x, cache(kv_heads=1), b, {}),
        "more heads": (layer(heads=8), x, c, b, {}),
        "a larger head": (layer(heads=2, kv_heads=1, dim=32), x, cache(1, 32), b, {}),
        "a larger hidden size": (layer(hidden=96), wide, c, b, dict(out=wide.clone())),
        "a cache of another type": (own, x, cache(dtype=torch.bfloat16), b, {}),
        "a cache of other heads": (own, x, cache(kv_heads=4), b, {}),
        "a cache of another head size": (own, x, cache(dim=32), b, {}),
        "a longer table": (own, x, c, batch(T, width=4000), {}),
        "other tokens": (own, x, c, batch(T + 1), {}),
        "x of another size": (own, wide, c, b, {}),
        "x of another type": (own, x.double(), c, b, {}),
        "x of other strides": (own, torch.zeros(64, T).t() if T > 1 else x.half(), c, b, {}),
        "out of another size": (own, x, c, b, dict(out=wide)),
        "resid of fewer rows": (own, x, c, b, dict(resid=torch.zeros(T + 1, 64)[:0])),
    }
    for name, (a, xx, cc, bb, kw) in cases.items():
        with pytest.raises(ValueError):
            buf.run(a, xx, cc, bb, **kw)
            pytest.fail(name)
        assert not launched, name
    own.q_norm = torch.ones(8)
    with pytest.raises(ValueError):
        buf.run(own, x, c, b)
    own.q_norm = None
    own.inv_freq = own.inv_freq.float()
    with pytest.raises(ValueError):
        buf.run(own, x, c, b)
    assert not launched
    buf.run(layer(), x, c, b)
    assert launched[-1] == "gemm" and "attn" in launched


def test_more_new_tokens_of_a_sequence(launched):
    """The same rows with a larger max_q need a larger workspace."""
    own, c = layer(), cache()
    few, many = batch(40, 1, 40, 200), batch(40, 40, 1, 200)
    size = {b: R.attn_workspace_bytes(c, b, 4) for b in (few, many)}
    small, large = sorted((few, many), key=size.get)
    assert size[small] < size[large]
    buf = R.AttentionBuffers(own, c, small, device="cpu")
    with pytest.raises(ValueError, match="workspace"):
        buf.run(own, torch.zeros(40, 64), c, large)
    assert not launched


@pytest.mark.parametrize("T", [3, 6])
def test_a_format_that_needs_more_workspace(T, launched):
    """Buffers for FP3 projections, a layer whose FP4 ones need more room."""
    small, large = layer(fmt=3), layer(fmt=4)
    for a in (small, large):
        a.need = max(R.gemm_workspace_bytes(W, T) for W in (a.wq, a.wk, a.wv, a.wo))
    buf = R.AttentionBuffers(small, cache(), batch(T), device="cpu")
    if large.need > small.need:
        with pytest.raises(ValueError, match="workspace"):
            buf.run(large, torch.zeros(T, 64), cache(), batch(T))
        assert not launched
    else:
        buf.run(large, torch.zeros(T, 64), cache(), batch(T))


def test_buffers_made_in_inference_mode(launched):
    with torch.inference_mode():
        own, c, b, x = layer(), cache(), batch(3), torch.zeros(3, 64)
        buf = R.AttentionBuffers(own, c, b, device="cpu")
        buf.run(own, x, c, b)
    buf.run(own, x, c, b)
    assert launched.count("attn") == 2


def test_layer_refuses_its_arguments():
    for kw in (dict(heads=4, kv_heads=3), dict(window=-1), dict(sinks=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            layer(**kw)
