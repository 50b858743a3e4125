"""CPU tests of the adapters' refusals: every bad argument fails before any
HIP call, and the binding checks tensors before it takes their addresses."""

import ctypes

import pytest
import torch

import bit_block_quantized_amd as R

INVAL, ALIGN, WORKSPACE = -1, -2, -5
P = 1 << 20  # an aligned address that is never followed


def status(mat=None, mats=1, ws=P, ws_bytes=1 << 30, **kw):
    m = R.LoraMatC(*{**dict(a=P, b=P, scale=P, resid=P, y=P, rows=100, reserved=0), **(mat or {})}.values())
    d = dict(type=R.BF16, n_adapters=4, rank=16, cols=64, n_tokens=0, n_mats=mats, x=P, x_stride=64, ids=P)
    c = R.LoraC(*{**d, **kw}.values(), (R.LoraMatC * R.LORA_MAX_MATS)(*[m] * min(mats, 4)))
    return R.lib().rfx_lora_apply(ctypes.byref(c), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(type=R.F32), INVAL), (dict(type=9), INVAL), (dict(n_adapters=0), INVAL), (dict(n_adapters=(1 << 20) + 1), INVAL),
    (dict(rank=0), INVAL), (dict(rank=12), INVAL), (dict(rank=136), INVAL), (dict(cols=0), INVAL), (dict(cols=48), INVAL),
    (dict(n_tokens=-1), INVAL), (dict(n_tokens=(1 << 19) + 1), INVAL), (dict(mats=0), INVAL), (dict(mats=5), INVAL),
    (dict(x=None), INVAL), (dict(x=P + 4), ALIGN), (dict(x_stride=60), INVAL), (dict(x_stride=66), INVAL),
    (dict(ids=None), INVAL), (dict(ids=P + 2), ALIGN), (dict(mat=dict(a=None)), INVAL), (dict(mat=dict(a=P + 8)), ALIGN),
    (dict(mat=dict(b=P + 2)), ALIGN), (dict(mat=dict(scale=P + 2)), ALIGN), (dict(mat=dict(resid=P + 1)), ALIGN),
    (dict(mat=dict(y=None)), INVAL), (dict(mat=dict(rows=0)), INVAL), (dict(mat=dict(rows=(1 << 24) + 1)), INVAL),
    (dict(n_tokens=1, ws=None), WORKSPACE), (dict(n_tokens=1, ws_bytes=16), WORKSPACE), (dict(n_tokens=1, ws=P + 64), ALIGN)])
def test_refuses(kw, want):
    assert status(**kw) == want


def test_takes():
    for kw in ({}, dict(mats=4), dict(mat=dict(scale=None, resid=None)), dict(type=R.F16, x_stride=72), dict(mat=dict(y=P + 4))):
        assert status(**kw) == 0
    assert R.lib().rfx_lora_apply(None, P, 1 << 30, None) == INVAL


def test_refuses_results_that_overlap():
    """Whole, in part, and the last row of one with the first of the next."""
    m = lambda y, rows: R.LoraMatC(P, P, None, None, y, rows, 0)  # noqa: E731
    for a, b in ((m(P, 8), m(P, 8)), (m(P, 8), m(P + 16, 4)), (m(P + 80, 64), m(P, 8)), (m(P, 1 << 24), m(P + (1 << 27), 4))):
        c = R.LoraC(R.BF16, 4, 16, 64, 3, 2, P, 64, P, (R.LoraMatC * R.LORA_MAX_MATS)(a, b))
        assert R.lib().rfx_lora_apply(ctypes.byref(c), None, 0, None) == INVAL
    c = R.LoraC(R.BF16, 4, 16, 64, 3, 2, P, 64, P, (R.LoraMatC * R.LORA_MAX_MATS)(m(P, 8), m(P + 96, 8)))  # neighbours
    assert R.lib().rfx_lora_apply(ctypes.byref(c), None, 0, None) == WORKSPACE


def test_packed_arguments_are_the_structure():
    m = R.LoraMatC(P, 2 * P, 3 * P, 4 * P, 5 * P, 77, 0)
    c = R.LoraC(R.F16, 3, 24, 96, 5, 2, 6 * P, 128, 7 * P, (R.LoraMatC * 4)(m, m))
    packed = R._pack_lora(R.F16, 3, 24, 96, 5, 2, 6 * P, 128, 7 * P) + 2 * R._pack_lora_mat(P, 2 * P, 3 * P, 4 * P, 5 * P, 77, 0)
    assert packed.ljust(ctypes.sizeof(R.LoraC), b"\0") == bytes(c)


def test_workspace_sizes():
    need = R.lib().rfx_lora_workspace_bytes
    assert need(1, 16, 1, 64, 4) > 0 and need(100, 16, 3, 64, 4) > need(100, 16, 1, 64, 4)
    for bad in ((-1, 16, 1, 64, 4), (1, 12, 1, 64, 4), (1, 16, 5, 64, 4), (1, 16, 1, 40, 4), (1, 16, 1, 64, 0)):
        assert need(*bad) == 0
    # a split has the padded tokens' sums: 17 tokens in 32, ranks of 40 in 48
    assert need(17, 40, 2, 256, 4) == 32 * 2 * 48 * 4 and need(17, 40, 2, 4096, 4) % need(17, 40, 2, 256, 4) == 0


def test_binding_checks_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    for a, b, scale in ((bf(2, 16, 64).float(), bf(2, 50, 16).float(), None), (bf(2, 16, 64), bf(2, 50, 16).half(), None),
                        (bf(2, 12, 64), bf(2, 50, 12), None), (bf(2, 16, 48), bf(2, 50, 16), None),
                        (bf(2, 16, 64), bf(3, 50, 16), None), (bf(2, 16, 64), bf(2, 50, 8), None),
                        (bf(2, 64, 16).transpose(1, 2), bf(2, 50, 64), None), (bf(2, 16, 64), bf(2, 50, 16), torch.zeros(3)),
                        (bf(2, 16, 64), bf(2, 50, 16), torch.zeros(2).double()), (bf(2, 136, 64), bf(2, 50, 136), None)):
        with pytest.raises(ValueError):
            R.DeviceLora(a, b, scale)
    one, other = R.DeviceLora(bf(2, 16, 64), bf(2, 50, 16)), R.DeviceLora(bf(2, 24, 64), bf(2, 50, 24))
    x, ids, y = torch.zeros(3, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 50)
    for bad in ((x.double(), ids, [one], [y]), (x[:2], ids, [one], [y]), (torch.zeros(3, 96), ids, [one], [y]),
                (x, ids.long(), [one], [y]), (x, ids, [one], [y[:2]]), (x, ids, [one], [torch.zeros(50, 3).t()]),
                (x, ids, [one, other], [y, y]), (x, ids, [one] * 5, [y] * 5), (x, ids, [one], [y, y]),
                (x, ids, [one], [y], [y, y]), (x, ids, [one], [y], [y.half()]), (x, ids, [one], [y])):  # the last: host memory
        with pytest.raises(ValueError):
            R.lora(*bad)
