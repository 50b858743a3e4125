"""CPU tests of the layer classes' refusals with norms, adapters, shared
prefixes and heads: what does not fit is refused before any entry point that
launches work has been called."""

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R
from test_host_attention_layer import batch, cache, layer

LAUNCHES = ("quantize_act", "gemv_grouped", "gemm", "qk_norm_rope", "attn", "attn_shared", "add_rms_norm", "lora")


@pytest.fixture
def launched(monkeypatch):
    calls = []
    for name in LAUNCHES:
        monkeypatch.setattr(R, name, lambda *a, _n=name, **k: calls.append(_n))
    monkeypatch.setattr(R.LogprobBuffers, "run", lambda self, *a, **k: calls.append("token_logprobs"))
    return calls


def adapters(rows, cols=64, rank=8, n=3, dtype=torch.bfloat16):
    return R.DeviceLora(torch.zeros(n, rank, cols, dtype=dtype), torch.zeros(n, rows, rank, dtype=dtype))


def prefix(n_groups=1, max_tokens=4, max_len=20):
    return R.KVPrefix(torch.zeros(n_groups + 1, dtype=torch.int32), torch.zeros(n_groups, dtype=torch.int32), max_tokens, max_len)


# hidden 64, four heads of 16 over two: 64, 32, 32 and 64 rows
FOUR = lambda **kw: [adapters(64, **kw), adapters(32, **kw), adapters(32, **kw), adapters(64, **kw)]  # noqa: E731


@pytest.mark.parametrize("T", [2, 6])
def test_attention_half_refuses(T, launched):
    own, c, b, p = layer(in_norm=np.ones(64)), cache(), batch(T), prefix()
    loras, ids, x = FOUR(), torch.zeros(T, dtype=torch.int32), torch.zeros(T, 64)
    buf = R.AttentionBuffers(own, c, b, device="cpu", prefix=p, loras=loras)
    plain = R.AttentionBuffers(own, c, b, device="cpu")
    windowed = layer(window=5)
    cases = {
        "a window beside a prefix": (buf, windowed, dict(prefix=p)),
        "three adapters": (buf, own, dict(loras=loras[:3], ids=ids)),
        "no adapter among them": (buf, own, dict(loras=[None] * 4, ids=ids)),
        "adapters without ids": (buf, own, dict(loras=loras)),
        "ids of another type": (buf, own, dict(loras=loras, ids=ids.long())),
        "ids of fewer tokens": (buf, own, dict(loras=loras, ids=ids[:1])),
        "rows of another matrix": (buf, own, dict(loras=[loras[1]] + loras[1:], ids=ids)),
        "columns of another": (buf, own, dict(loras=loras[:3] + [adapters(64, 96)], ids=ids)),
        "two ranks for one input": (buf, own, dict(loras=[adapters(64, rank=16)] + loras[1:], ids=ids)),
        "two types for one input": (buf, own, dict(loras=[adapters(64, dtype=torch.float16)] + loras[1:], ids=ids)),
        "a larger rank": (buf, own, dict(loras=FOUR(rank=64), ids=ids)),
        "buffers made without adapters": (plain, own, dict(loras=loras, ids=ids)),
    }
    for name, (buffers, a, kw) in cases.items():
        with pytest.raises(ValueError):
            buffers.run(a, x, c, b, **kw)
            pytest.fail(name)
        assert not launched, name
    own.in_norm = torch.ones(63)
    with pytest.raises(ValueError):
        buf.run(own, x, c, b)
    assert not launched
    own.in_norm = torch.ones(64)
    buf.run(own, x, c, b, prefix=p, loras=loras, ids=ids)
    assert launched[0] == "add_rms_norm" and launched[-2:] == ["gemm", "lora"]
    assert "attn_shared" in launched and "attn" not in launched and launched.count("lora") == 2
    del launched[:]
    buf.run(own, x, c, b, loras=[None, None, None, loras[3]], ids=ids)
    assert launched.count("lora") == 1 and launched[-1] == "lora" and "attn" in launched


def test_larger_prefixes_need_larger_buffers(launched):
    own, c, b = layer(), cache(), batch(2, seqs=2, width=400)
    small, large = prefix(max_len=10), prefix(n_groups=8, max_tokens=64, max_len=6000)
    sizes = [R.attn_shared_workspace_bytes(c, b, p, 4) for p in (small, large)]
    assert sizes[0] < sizes[1]
    buf = R.AttentionBuffers(own, c, b, device="cpu", prefix=small)
    with pytest.raises(ValueError, match="workspace"):
        buf.run(own, torch.zeros(2, 64), c, b, prefix=large)
    assert not launched


@pytest.mark.parametrize("q", [1, 7])
def test_head_refuses(q, launched):
    head = lambda V=100, H=64, **kw: R.DeviceHead.build(V, H, np.ones((V, H), np.float32), device="cpu", **kw)  # noqa: E731
    own = head(norm=np.ones(64))
    buf = R.HeadBuffers(own, q, 5, device="cpu")
    x, t = torch.zeros(q, 64), torch.zeros(q, dtype=torch.int32)
    other = head()
    other.norm = torch.ones(32)
    for name, (h, xx, tt) in {"another vocabulary": (head(V=101), x, t), "another hidden size": (head(H=96), x, t),
                              "rows of another size": (own, torch.zeros(q, 96), t), "more rows": (own, torch.zeros(q + 1, 64), t),
                              "another type": (own, x.double(), t), "tokens of another type": (own, x, t.long()),
                              "more tokens": (own, x, torch.zeros(q + 1, dtype=torch.int32)), "a shorter norm": (other, x, t)}.items():
        with pytest.raises(ValueError):
            buf.run(h, xx, tt)
            pytest.fail(name)
        assert not launched, name
    buf.run(own, x, t)
    assert launched == ["add_rms_norm", "gemm", "token_logprobs"]
    buf.run(head(), x)
    assert launched[3:] == ["quantize_act", "gemm", "token_logprobs"]
    with pytest.raises(ValueError):
        R.DeviceHead(own.w, eps=-1.0)
