"""CPU tests of the refusals of the residual norm and of the log
probabilities: every bad argument fails before any HIP call, and the binding
checks tensors before it takes their addresses."""

import ctypes
import math

import pytest
import torch

import bit_block_quantized_amd as R

INVAL, ALIGN, WORKSPACE = -1, -2, -5
P = 1 << 20  # an aligned address that is never followed


def norm_status(**kw):
    d = dict(x=P, delta=P, x_stride=64, delta_stride=64, weight=P, sum=P, y=None, xq=P, xs=P, xsum=P, eps=1e-6, q=0,
             cols=64, reserved=0)
    return R.lib().rfx_add_rms_norm(ctypes.byref(R.NormC(*{**d, **kw}.values())), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=-1), INVAL), (dict(q=(1 << 21) + 1), INVAL), (dict(cols=0), INVAL), (dict(cols=48), INVAL),
    (dict(cols=(1 << 20) + 32), INVAL), (dict(eps=-1e-6), INVAL), (dict(eps=math.nan), INVAL), (dict(eps=math.inf), INVAL),
    (dict(x_stride=60), INVAL), (dict(x_stride=66), INVAL), (dict(delta_stride=0), INVAL), (dict(x=None), INVAL),
    (dict(x=P + 4), ALIGN), (dict(delta=P + 8), ALIGN), (dict(weight=P + 4), ALIGN), (dict(sum=P + 4), ALIGN),
    (dict(y=P + 8, sum=None), ALIGN), (dict(xq=P + 4), ALIGN), (dict(xs=None), INVAL), (dict(xsum=P + 2), ALIGN),
    (dict(sum=None, xq=None), INVAL), (dict(y=P), INVAL)])
def test_norm_refuses(kw, status):
    assert norm_status(**kw) == status


def test_norm_takes():
    for kw in ({}, dict(delta=None, delta_stride=0), dict(weight=None), dict(xq=None, xs=None, xsum=None),
               dict(sum=None, y=P), dict(x_stride=1 << 20)):
        assert norm_status(**kw) == 0
    assert R.lib().rfx_add_rms_norm(None, None) == INVAL


def test_packed_norm_arguments_are_the_structure():
    a = R.NormC(P, 2 * P, 128, 192, 3 * P, 4 * P, 0, 5 * P, 6 * P, 7 * P, 1e-5, 3, 64, 0)
    assert R._pack_norm(P, 2 * P, 128, 192, 3 * P, 4 * P, 0, 5 * P, 6 * P, 7 * P, 1e-5, 3, 64, 0) == bytes(a)


def test_norm_binding_checks_tensors():
    f = lambda *s: torch.zeros(s)  # noqa: E731
    codes = dict(xq=torch.zeros(2, 64, dtype=torch.int8), xs=f(2, 2), xsum=torch.zeros(2, 2, dtype=torch.int32))
    ok = dict(x=f(2, 64), weight=f(64), eps=1e-6, delta=f(2, 64), out=f(2, 64), y=f(2, 64), **codes)
    for name, bad in (("x", f(2, 64).double()), ("x", f(64, 2).t()), ("weight", f(63)), ("weight", f(64).half()),
                      ("delta", f(1, 64)), ("out", f(2, 128)[:, ::2]), ("y", f(2, 128)[:, :64]), ("xq", f(2, 64)),
                      ("xs", f(2, 1)), ("xsum", f(2, 2)), ("xq", None), ("x", f(2, 64))):  # the last: host memory
        with pytest.raises(ValueError):
            R.add_rms_norm(**{**ok, name: bad})


def logp_status(stride=100, logits=P, tokens=P, ws=P, ws_bytes=1 << 30, **kw):
    d = dict(type=R.F32, q=0, n_vocab=100, top_k=4, logprob=P, lse=P, entropy=P, rank=P, top_index=P, top_logprob=P)
    return R.lib().rfx_token_logprobs(logits, stride, tokens, ctypes.byref(R.LogprobC(*{**d, **kw}.values())), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), INVAL), (dict(type=-1), INVAL), (dict(q=-1), INVAL), (dict(q=65537), INVAL), (dict(n_vocab=0), INVAL),
    (dict(n_vocab=(1 << 19) + 1, stride=1 << 20), INVAL), (dict(top_k=-1), INVAL), (dict(top_k=65), INVAL),
    (dict(stride=99), INVAL), (dict(stride=-100), INVAL), (dict(logits=None), INVAL), (dict(logits=P + 2), ALIGN),
    (dict(logits=P + 1, type=R.BF16), ALIGN), (dict(tokens=None), INVAL), (dict(tokens=P + 2), ALIGN),
    (dict(top_k=0), INVAL), (dict(lse=P + 1), ALIGN), (dict(top_index=P + 2), ALIGN),
    (dict(logprob=None, lse=None, entropy=None, rank=None, top_index=None, top_logprob=None), INVAL),
    (dict(q=1, ws=None), WORKSPACE), (dict(q=1, ws_bytes=64), WORKSPACE), (dict(q=1, ws=P + 16), ALIGN)])
def test_logprobs_refuses(kw, status):
    assert logp_status(**kw) == status


def test_logprobs_takes():
    assert logp_status() == 0
    assert logp_status(tokens=None, logprob=None, rank=None) == 0
    assert logp_status(top_k=0, top_index=None, top_logprob=None) == 0
    assert logp_status(type=R.BF16, logits=P + 2) == 0
    assert R.lib().rfx_token_logprobs(P, 100, P, None, P, 1 << 30, None) == INVAL


def test_logprobs_workspace_sizes():
    need = R.token_logprobs_workspace_bytes
    assert need(1, 100, 0) >= 32 and need(1, 100, 0) % 256 == 0
    assert need(4, 1000, 64) > need(4, 1000, 0)
    assert need(-1, 100, 0) == need(1, 0, 0) == need(1, 100, 65) == need(1, (1 << 19) + 1, 0) == 0
    assert need(65536, 1 << 19, 64) > 1 << 31
    with pytest.raises(ValueError, match="below 2"):
        need(1 << 32, 100, 0)


def test_logprob_buffers_check_tensors():
    for bad in (dict(q=0, n_vocab=10), dict(q=1, n_vocab=0), dict(q=1, n_vocab=10, top_k=65), dict(q=65537, n_vocab=10)):
        with pytest.raises(ValueError):
            R.LogprobBuffers(device="cpu", **bad)
    b = R.LogprobBuffers(2, 50, 3, device="cpu")
    z, t = torch.zeros(2, 50), torch.zeros(2, dtype=torch.int32)
    for bad in ((z.double(), t), (z[:1], t), (torch.zeros(50, 2).t(), t), (torch.zeros(2, 100)[:, ::2], t), (z, t.long()),
                (z, t[:1]), (z, t)):  # the last: host memory
        with pytest.raises(ValueError):
            b.run(*bad)
