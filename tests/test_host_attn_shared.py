"""CPU tests of rfx_attn_shared's refusals: every bad argument fails before any
HIP call, and the binding checks tensors before it takes their addresses."""

import ctypes
import math

import pytest
import torch

import bit_block_quantized_amd as R
from test_host_attn import BAD_BATCH, BAD_CACHE, ALIGN, INVAL, WORKSPACE, P, batch, cache


def prefix(**kw):
    d = dict(n_groups=1, max_tokens=4, max_len=100, reserved=0, seq_off=P, len=P)
    return R.KVPrefixC(*{**d, **kw}.values())


def status(c=None, b=None, p=None, heads=8, scale=0.125, q=P, out=P, out_type=R.F32, ws=P, ws_bytes=1 << 30):
    c, b, p = c or cache(), b or batch(n_tokens=0), p or prefix()
    return R.lib().rfx_attn_shared(q, ctypes.byref(c), ctypes.byref(b), ctypes.byref(p), heads, scale, out, out_type, ws,
                                   ws_bytes, None)


def test_bad_descriptors():
    for kw, want, word in BAD_CACHE:
        assert status(c=cache(**kw)) == want and word in R.lib().rfx_last_error().decode()
    for kw, want, word in BAD_BATCH:
        assert status(b=batch(**kw)) == want and word in R.lib().rfx_last_error().decode()
    for kw, want in ((dict(n_groups=0), INVAL), (dict(n_groups=(1 << 23) + 1), INVAL), (dict(max_tokens=0), INVAL),
                     (dict(max_tokens=(1 << 23) + 1), INVAL), (dict(max_len=0), INVAL), (dict(seq_off=None), INVAL),
                     (dict(seq_off=P + 2), ALIGN), (dict(len=None), INVAL), (dict(len=P + 1), ALIGN)):
        assert status(p=prefix(**kw)) == want, kw
    L = R.lib()
    assert L.rfx_attn_shared(P, ctypes.byref(cache()), ctypes.byref(batch()), None, 8, 0.1, P, 0, P, 1 << 30, None) == INVAL
    assert L.rfx_attn_shared(P, None, ctypes.byref(batch()), ctypes.byref(prefix()), 8, 0.1, P, 0, P, 1 << 30, None) == INVAL


@pytest.mark.parametrize("max_q", [2, 100]) # the second goes to rfx_attn
def test_bad_arguments(max_q):
    for kw, want in ((dict(heads=0), INVAL), (dict(heads=7), INVAL), (dict(scale=0.0), INVAL), (dict(scale=math.inf), INVAL),
                     (dict(scale=math.nan), INVAL), (dict(scale=1.5 * 2.0 ** 127), INVAL), (dict(out_type=R.F16), INVAL),
                     (dict(q=None), INVAL), (dict(q=P + 4), ALIGN), (dict(out=None), INVAL), (dict(out=P + 8), ALIGN),
                     (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(ws=P + 16), ALIGN)):
        assert status(b=batch(max_q=max_q, table_stride=1000, n_tokens=0), **kw) == want, kw


def test_workspace_sizes():
    need = R.lib().rfx_attn_shared_workspace_bytes

    def size(c=None, b=None, p=None, heads=8):
        return need(ctypes.byref(c or cache()), ctypes.byref(b or batch()), ctypes.byref(p or prefix()), heads)

    assert size() > 0 and size() % 256 == 0
    assert size(p=prefix(max_len=100000), b=batch(table_stride=10000)) > size(b=batch(table_stride=10000))
    assert size(p=prefix(n_groups=0)) == size(heads=7) == size(c=cache(head_dim=0)) == size(b=batch(n_seq=0)) == 0
    many = batch(max_q=100, table_stride=1000)
    assert size(b=many) == R.lib().rfx_attn_workspace_bytes(ctypes.byref(cache()), ctypes.byref(many), 8)
    assert status(ws_bytes=size(b=batch(n_tokens=0)) - 1) == WORKSPACE
    assert status() == 0


def test_binding_checks_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in (lambda: R.KVPrefix(i(2), i(2), 4, 10), lambda: R.KVPrefix(i(3).long(), i(2), 4, 10),
                lambda: R.KVPrefix(i(3), i(2).float(), 4, 10), lambda: R.KVPrefix(i(6)[::2], i(2), 4, 10),
                lambda: R.KVPrefix(i(3), i(2), 1 << 31, 10), lambda: R.KVPrefix(i(3), i(2), 4, 1 << 32)):
        with pytest.raises(ValueError):
            bad()
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    c, b, p = R.DeviceKVCache(k, k.clone()), R.KVBatch(i(3), i(2), i(2, 4), 2, 1), R.KVPrefix(i(3), i(2), 4, 10)
    q, o = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 64))
    for bad in ((q.half(), o), (q[:1], o), (q, o.double()), (q, o.transpose(0, 1)), (q, o)):  # the last: host memory
        with pytest.raises(ValueError):
            R.attn_shared(bad[0], c, b, p, bad[1], 0.1)
