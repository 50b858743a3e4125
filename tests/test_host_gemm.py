"""CPU tests of rfx_gemm's refusals and workspace sizes: every bad argument
fails before any HIP call."""

import contextlib
import ctypes

import pytest
import torch

import bit_block_quantized_amd as R

INVAL, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -4, -5
P = 1 << 20  # an aligned address that is never followed


def status(q=4, act=0, xq=P, xs=P, xsum=P, bias=None, resid=None, y=P, ws=None, ws_bytes=0, **kw):
    W = R.QMat(*{**dict(fmt=4, rows=1024, cols=4096, count=1, data=P), **kw}.values())
    return R.lib().rfx_gemm(ctypes.byref(W), xq, xs, xsum, q, bias, act, resid, y, ws, ws_bytes, None)


def need(q, **kw):
    W = R.QMat(*{**dict(fmt=4, rows=1024, cols=4096, count=1, data=P), **kw}.values())
    return R.lib().rfx_gemm_workspace_bytes(ctypes.byref(W), q)


def test_refusals():
    for kw, st in ((dict(fmt=5), INVAL), (dict(rows=0), INVAL), (dict(cols=48), INVAL), (dict(count=2), INVAL),
                   (dict(data=None), INVAL), (dict(data=P + 128), ALIGN), (dict(q=0), INVAL), (dict(q=65537), INVAL),
                   (dict(act=-1), INVAL), (dict(act=5), INVAL), (dict(xq=None), INVAL), (dict(xq=P + 8), ALIGN),
                   (dict(xs=P + 2), ALIGN), (dict(xsum=None), INVAL), (dict(y=None), INVAL), (dict(y=P + 1), ALIGN),
                   (dict(bias=P + 2), ALIGN), (dict(resid=P + 3), ALIGN), (dict(ws=None), WORKSPACE),
                   (dict(q=9, fmt=8), UNSUPPORTED), (dict(q=9, fmt=12), UNSUPPORTED), (dict(q=9, fmt=16), UNSUPPORTED),
                   (dict(q=9, fmt=13), UNSUPPORTED), (dict(q=9), WORKSPACE),
                   (dict(q=9, ws=P, ws_bytes=need(9) - 1), WORKSPACE), (dict(q=9, ws=P + 64, ws_bytes=1 << 40), ALIGN)):
        assert status(**kw) == st, kw
    assert R.lib().rfx_gemm(None, P, P, P, 1, None, 0, None, P, None, 0, None) == INVAL


def test_workspace_sizes():
    W = R.QMat(4, 1024, 4096, 1, P)
    for q in (1, 4):
        assert need(q) == R.lib().rfx_gemv_workspace_bytes(ctypes.byref(W), q) > 0
    # the first 256 KiB stay the GEMV form's, whose slots fit in them
    for q in (5, 64, 2048, 65536):
        assert need(q) > (256 << 10) + 2 * q * 4096
    assert all(R.lib().rfx_gemv_workspace_bytes(ctypes.byref(R.QMat(4, r, c, 1, P)), 4) <= 256 << 10
               for r in (1, 64, 777, 4096, 20000) for c in (32, 512, 4096, 65536))
    assert need(0) == need(65537) == need(9, fmt=8) == need(9, cols=33) == 0


def test_weights_in_host_memory_are_refused():
    W = R.DeviceQMat(4, 64, 32, torch.zeros(8704, dtype=torch.uint8))
    with pytest.raises(ValueError, match="host memory"):
        R.gemm(W, P, P, P, 1, P)


def test_weights_on_another_device(monkeypatch):
    """The call runs with W's device current, on that device's stream."""
    calls, entered = [], []

    class Lib:
        @staticmethod
        def rfx_gemm(*args):
            calls.append((list(entered), args[-1]))
            return 0

    @contextlib.contextmanager
    def guard(index):
        entered.append(index)
        yield
        entered.pop()

    t = R._torch()
    monkeypatch.setattr(R, "lib", lambda: Lib)
    monkeypatch.setattr(t, "current_device", lambda: entered[-1] if entered else 0)
    monkeypatch.setattr(t, "device_guard", guard)
    monkeypatch.setattr(t, "raw_stream", lambda index: 100 + index)
    W = R.DeviceQMat(4, 64, 32, P)
    for index, stream in ((3, None), (0, None), (3, 7), (None, None)):
        W.index = index
        R.gemm(W, P, P, P, 1, P, stream=stream)
    assert calls == [([3], 103), ([], 100), ([3], 7), ([], 100)]


def test_slots_of_every_shape_fit_in_front_of_the_operands():
    """A workspace's first part is the GEMV form's, whatever its shape: what a
    call with more columns reserves in front of its operands (here one K tile
    of one column tile, FP2: 8 KiB of codes and 512 bytes of scales) holds the
    exchange slots of every matrix with four columns."""
    reserved = need(5, fmt=2, rows=1, cols=32) - 8192 - 512
    most = max(need(4, rows=rows, cols=cols) for rows in range(1, 64 * 400, 64) for cols in (512, 1024, 2048, 4096, 8192, 1 << 20))
    assert most == 47 * 7 * 4 * 256
    assert most <= reserved


@pytest.mark.parametrize("q", [3, 40])
def test_binding_checks_tensors(q, monkeypatch):
    """Tensors of another type, size, layout or device are refused before the
    call; larger ones (a buffer's first rows) and bare addresses are taken."""
    calls = []

    class Lib:
        @staticmethod
        def rfx_gemm(*args):
            calls.append(args)
            return 0

    W = R.DeviceQMat(4, 100, 64, torch.zeros(1, dtype=torch.uint8))
    ok = dict(xq=torch.zeros(q, 64, dtype=torch.int8), xs=torch.zeros(q, 2), xsum=torch.zeros(q, 2, dtype=torch.int32), q=q,
              y=torch.zeros(q, 100), bias=torch.zeros(100), resid=torch.zeros(q, 100), ws=torch.zeros(256, dtype=torch.uint8))
    bad = [dict(xq=ok["xq"].to(torch.uint8)), dict(xq=ok["xq"][:-1]), dict(xq=torch.zeros(64, q, dtype=torch.int8).t()),
           dict(xs=ok["xs"].double()), dict(xs=ok["xs"][:, :1]), dict(xs=torch.zeros(2, q).t()),
           dict(xsum=ok["xsum"].long()), dict(xsum=ok["xsum"][1:]), dict(y=ok["y"].half()), dict(y=ok["y"][1:]),
           dict(y=torch.zeros(100, q).t()), dict(y=torch.zeros(q, 200)[:, ::2]), dict(bias=ok["bias"][:99]),
           dict(bias=ok["bias"].bfloat16()), dict(bias=torch.zeros(200)[::2]), dict(resid=ok["resid"][1:]),
           dict(resid=ok["resid"].double()), dict(resid=torch.zeros(100, q).t()), dict(resid=torch.zeros(100).expand(q, 100)),
           dict(ws=torch.zeros(512, dtype=torch.uint8)[::2])]
    monkeypatch.setattr(R, "lib", lambda: Lib)
    monkeypatch.setattr(R, "_call_on", lambda index, stream, fn, *args: fn(*args))
    for kw in bad:
        with pytest.raises(ValueError, match=next(iter(kw))):
            R.gemm(W, **{**ok, **kw})
    W.index = 3
    for name in ok:
        if name != "q": # the others are where the weights are
            monkeypatch.setattr(torch.Tensor, "get_device", lambda t, _bad=ok[name]: 2 if t is _bad else 3)
            with pytest.raises(ValueError, match=name):
                R.gemm(W, **ok)
    assert not calls
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 3)
    R.gemm(W, **ok)
    R.gemm(W, **{**ok, "xq": torch.zeros(q + 5, 64, dtype=torch.int8), "y": torch.zeros(q, 10, 10), "bias": None, "resid": None,
                 "ws": None})
    R.gemm(W, P, P, P, q, P, resid=P)
    assert len(calls) == 3 and calls[0][8] == ok["y"].data_ptr() and calls[1][9:] == (None, 0)
    assert calls[2][1:4] == (P, P, P) and calls[2][7:9] == (P, P)


def test_weights_that_only_have_an_address():
    """data may be any object with data_ptr(), an address or None."""
    class Block:
        @staticmethod
        def data_ptr():
            return P

    assert [R.DeviceQMat(4, 64, 32, d).index for d in (Block(), P, None)] == [None] * 3
    assert R.DeviceQMat(4, 64, 32, Block()).c.data == P
    assert R.DeviceQMat(4, 64, 32, torch.zeros(8704, dtype=torch.uint8)).index == -1


@pytest.mark.parametrize("fmt", [2, 3, 4])
def test_matrices_past_the_kernels_32_bit_numbers(fmt):
    """Rows that do not fit 32 bits once rounded up, and K tiles times splits
    past 2^31, are refused."""
    for kw in (dict(rows=(1 << 30) + 1), dict(rows=(1 << 31) - 1, cols=32), dict(cols=(1 << 29) + 32, rows=1)):
        assert need(5, fmt=fmt, **kw) == 0 and status(q=5, fmt=fmt, ws=P, ws_bytes=1 << 60, **kw) == UNSUPPORTED, kw
    assert need(5, fmt=fmt, rows=1 << 30, cols=32) > 0 < need(5, fmt=fmt, rows=1, cols=1 << 29)
