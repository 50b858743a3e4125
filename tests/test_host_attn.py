"""CPU tests of the paged-attention entry points' refusals: every bad
argument fails before any HIP call, with its status and a message that names
it, and the binding checks tensors before it takes their addresses."""

import ctypes
import math

import pytest
import torch

import bit_block_quantized_amd as R

INVAL, ALIGN, WORKSPACE = -1, -2, -5
P = 1 << 20  # an aligned address that is never followed


def cache(**kw):
    d = dict(type=R.BF16, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, reserved=0, k=P, v=P)
    return R.KVCacheC(*{**d, **kw}.values())


def batch(**kw):
    d = dict(n_seq=2, n_tokens=4, max_q=2, table_stride=8, q_off=P, kv_len=P, page_table=P)
    return R.KVBatchC(*{**d, **kw}.values())


def rope(**kw):
    d = dict(q=P, k=P, v=P, q_stride=512, k_stride=128, v_stride=128, inv_freq=P, q_weight=P, k_weight=None, eps=1e-6,
             n_heads=8, rot_dim=64, interleaved=0)
    return R.QkRopeC(*{**d, **kw}.values())


def attn_status(c, b, heads=8, scale=0.125, window=0, sinks=0, q=P, out=P, out_type=R.F32, ws=P, ws_bytes=1 << 30):
    return R.lib().rfx_attn(q, ctypes.byref(c), ctypes.byref(b), heads, scale, window, sinks, out, out_type, ws, ws_bytes, None)


def rope_status(a, c, b, out=P):
    return R.lib().rfx_qk_norm_rope(ctypes.byref(a), ctypes.byref(c), ctypes.byref(b), out, None)


BAD_CACHE = [(dict(type=R.F32), INVAL, "type"), (dict(type=7), INVAL, "type"), (dict(head_dim=0), INVAL, "head_dim"),
             (dict(head_dim=60), INVAL, "head_dim"), (dict(head_dim=264), INVAL, "head_dim"),
             (dict(n_kv_heads=0), INVAL, "heads"), (dict(n_kv_heads=3), INVAL, "heads"),
             (dict(page_size=0), INVAL, "page_size"), (dict(page_size=24), INVAL, "page_size"),
             (dict(page_size=8192), INVAL, "page_size"), (dict(n_pages=0), INVAL, "n_pages"),
             (dict(k=None), INVAL, "cache k"), (dict(v=P + 8), ALIGN, "cache v")]
BAD_BATCH = [(dict(n_seq=0), INVAL, "n_seq"), (dict(n_tokens=-1), INVAL, "n_tokens"), (dict(max_q=0), INVAL, "max_q"),
             (dict(n_tokens=(1 << 23) + 1), INVAL, "n_tokens"), (dict(max_q=(1 << 23) + 1), INVAL, "max_q"),
             (dict(table_stride=0), INVAL, "table_stride"), (dict(table_stride=(1 << 26) + 1), INVAL, "table_stride"),
             (dict(q_off=None), INVAL, "q_off"), (dict(kv_len=P + 2), ALIGN, "kv_len"), (dict(page_table=None), INVAL, "page_table")]


@pytest.mark.parametrize("call", ["attn", "rope"])
def test_bad_descriptors(call):
    for which, cases in (("c", BAD_CACHE), ("b", BAD_BATCH)):
        for kw, status, word in cases:
            c, b = cache(**kw) if which == "c" else cache(), batch(**kw) if which == "b" else batch()
            st = attn_status(c, b) if call == "attn" else rope_status(rope(), c, b)
            assert st == status, (kw, st)
            assert word in R.lib().rfx_last_error().decode(), (kw, R.lib().rfx_last_error())
    L = R.lib()
    assert L.rfx_attn(P, None, ctypes.byref(batch()), 8, 0.125, 0, 0, P, 0, P, 1 << 30, None) == INVAL
    assert L.rfx_qk_norm_rope(None, ctypes.byref(cache()), ctypes.byref(batch()), P, None) == INVAL


def test_bad_attention_arguments():
    for kw, status in ((dict(heads=0), INVAL), (dict(heads=7), INVAL), (dict(heads=2048), INVAL), (dict(scale=0.0), INVAL),
                       (dict(scale=-1.0), INVAL), (dict(scale=math.inf), INVAL), (dict(scale=math.nan), INVAL),
                       (dict(window=-1), INVAL), (dict(sinks=-1), INVAL), (dict(out_type=R.F16), INVAL),
                       (dict(out_type=9), INVAL), (dict(q=None), INVAL), (dict(q=P + 4), ALIGN), (dict(out=None), INVAL),
                       (dict(out=P + 8), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
                       (dict(ws=P + 16), ALIGN)):
        # a table long enough that the keys are split and a workspace is needed
        assert attn_status(cache(), batch(table_stride=1000), **kw) == status, kw


def test_bad_rope_arguments():
    for kw, status in ((dict(rot_dim=-8), INVAL), (dict(rot_dim=72), INVAL), (dict(rot_dim=12), INVAL),
                       (dict(eps=-1.0), INVAL), (dict(eps=math.nan), INVAL), (dict(n_heads=3), INVAL),
                       (dict(q_stride=508), INVAL), (dict(q_stride=514), INVAL), (dict(k_stride=124), INVAL),
                       (dict(v_stride=0), INVAL), (dict(q=None), INVAL), (dict(k=P + 4), ALIGN), (dict(v=None), INVAL),
                       (dict(inv_freq=None), INVAL), (dict(inv_freq=P + 4), ALIGN), (dict(q_weight=P + 4), ALIGN),
                       (dict(k_weight=P + 8), ALIGN)):
        assert rope_status(rope(**kw), cache(), batch()) == status, kw
    assert rope_status(rope(), cache(), batch(), out=None) == INVAL


def test_no_tokens_is_nothing_to_do():
    assert attn_status(cache(), batch(n_tokens=0)) == 0
    assert rope_status(rope(), cache(), batch(n_tokens=0)) == 0


def test_workspace_sizes():
    L = R.lib()

    def need(c, b, heads):
        return L.rfx_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads)

    one = need(cache(), batch(n_seq=1, max_q=1, table_stride=1000), 8)
    assert one > 0 and one % 256 == 0
    # enough sequences fill the chip unsplit
    assert need(cache(), batch(n_seq=600, max_q=1, table_stride=1000), 8) == 0
    assert need(cache(head_dim=0), batch(), 8) == 0 and need(cache(), batch(n_seq=0), 8) == 0
    st = attn_status(cache(), batch(n_seq=1, max_q=1, table_stride=1000), ws_bytes=one - 1)
    assert st == WORKSPACE and str(one) in R.lib().rfx_last_error().decode()


def test_binding_checks_tensors():
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    c = R.DeviceKVCache(k, k.clone())
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = R.KVBatch(i(3), i(2), i(2, 4), 2, 1)
    q, o = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 64))
    for bad in (lambda: R.DeviceKVCache(k.float(), k.float()), lambda: R.DeviceKVCache(k, k[:2]),
                lambda: R.DeviceKVCache(k.transpose(1, 2), k.transpose(1, 2)), lambda: R.DeviceKVCache(k, k.half()),
                lambda: R.KVBatch(i(2), i(2), i(2, 4), 2, 1), lambda: R.KVBatch(i(3).long(), i(2), i(2, 4), 2, 1),
                lambda: R.KVBatch(i(3), i(2), i(4, 2).t(), 2, 1),
                lambda: R.attn(q.half(), c, b, o, 0.1), lambda: R.attn(q[:1], c, b, o, 0.1),
                lambda: R.attn(q, c, b, o.double(), 0.1), lambda: R.attn(q, c, b, o.transpose(0, 1), 0.1),
                lambda: R.attn(q, c, b, o, 0.1)):  # the last: host memory
        with pytest.raises(ValueError):
            bad()
    f = torch.zeros((2, 8, 64))
    inv = torch.zeros(32, dtype=torch.float64)
    ok = (f[:, :4], f[:, 4:6], f[:, 6:], c, b, q, inv)
    for j, x in ((0, f[:, :4].double()), (0, f[:1, :4]), (1, f[:, :4]), (2, f[:, ::4]), (5, q.half()), (6, inv.float())):
        with pytest.raises(ValueError):
            R.qk_norm_rope(*[x if n == j else a for n, a in enumerate(ok)])
    with pytest.raises(ValueError):
        R.qk_norm_rope(*ok, q_weight=torch.zeros(63))


def test_rope_inv_freq():
    f = R.rope_inv_freq(8, 16.0)
    assert f.tolist() == [1.0, 0.5, 0.25, 0.125]


def test_binding_refuses_windows_past_32_bits():
    c = R.DeviceKVCache(*(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    b = R.KVBatch(torch.tensor([0, 1], dtype=torch.int32), torch.tensor([1], dtype=torch.int32),
                  torch.zeros(1, 4, dtype=torch.int32), 1, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for kw in (dict(window=1 << 32), dict(window=5, sinks=(1 << 31) + 7)):
        with pytest.raises(ValueError, match="below 2"):
            R.attn(q, c, b, torch.zeros(1, 4, 64), 0.125, **kw)


def test_packed_rope_arguments_are_the_structure():
    a = rope(q_stride=520, k_stride=136, v_stride=144, eps=1e-5, n_heads=12, rot_dim=40, interleaved=True)
    packed = R._pack_qk_rope(P, P, P, 520, 136, 144, P, P, 0, 1e-5, 12, 40, True)
    assert packed == bytes(a) and len(packed) == ctypes.sizeof(R.QkRopeC)


def test_scale_that_overflows_with_log2_e():
    assert attn_status(cache(), batch(n_tokens=0), scale=1.5 * 2.0 ** 127) == INVAL
    assert attn_status(cache(), batch(n_tokens=0), scale=2.0 ** 127) == 0


@pytest.mark.parametrize("value", [-(1 << 31) - 1, -(1 << 32) + 5, 1 << 31, (1 << 32) + 5])
def test_binding_refuses_what_wraps_in_32_bits(value):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c, b, q, o = R.DeviceKVCache(k, k.clone()), R.KVBatch(i(2), i(1), i(1, 4), 1, 1), torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 64)
    for bad in (lambda: R.attn(q, c, b, o, 0.125, window=value), lambda: R.attn(q, c, b, o, 0.125, window=5, sinks=value),
                lambda: R.KVBatch(i(2), i(1), i(1, 4), value, 1), lambda: R.KVBatch(i(2), i(1), i(1, 4), 1, value)):
        with pytest.raises(ValueError, match="below 2"):
            bad()
