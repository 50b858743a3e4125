"""rfx_add_rms_norm against its definition in 64 bits: y is the fp32 number
next to it, the sum one fp32 addition, and codes, scales and code sums those
of y, bit for bit; scales are within a step of rfx_quantize_act's."""

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -20


def rows(q, cols, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(q, cols, generator=g)
    if spread and q:
        x *= 10.0 ** torch.linspace(-6, 4, q)[:, None]
        x[:, :: max(1, cols // 5)] *= 30
    return x


def outputs(q, cols):
    return dict(out=torch.full((q, cols), 7.0, device="cuda"), y=torch.full((q, cols), 7.0, device="cuda"),
                xq=torch.full((q, cols), 99, dtype=torch.int8, device="cuda"), xs=torch.full((q, cols // 32), 7.0, device="cuda"),
                xsum=torch.full((q, cols // 32), 99, dtype=torch.int32, device="cuda"))


def exact(x, delta, w, eps):
    h = x if delta is None else x + delta # one fp32 addition
    d = h.double()
    ms = d.square().mean(-1, keepdim=True) + float(np.float32(eps))
    y = d / torch.sqrt(torch.where(ms == 0, 1.0, ms))
    return h, y if w is None else y * w.double()


def quantized(y):
    """Codes, scales and code sums of fp32 rows, IEEE operations throughout."""
    b = y.reshape(len(y), -1, 32)
    s = np.abs(b).max(-1) * (np.float32(1) / np.float32(127))
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] == 0, 0, np.clip(np.rint(b / s[..., None]), -127, 127))
    return c.astype(np.int8).reshape(y.shape), s, c.sum(-1).astype(np.int32)


def check(o, h, y):
    got = {k: v.cpu() for k, v in o.items() if v is not None}
    if "out" in got:
        assert torch.equal(got["out"], h)
    if "y" in got:
        # half a step, and the fp64 arithmetic's own 2^-48 (sums of up to 2^20 squares: 2^-53 each, at random)
        tol = y.abs() * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -149
        assert ((got["y"].double() - y).abs() <= tol).all()
    if "xq" in got:
        src = got["y"] if "y" in got else y.float()
        for name, want in zip(("xq", "xs", "xsum"), quantized(src.numpy())):
            assert np.array_equal(got[name].numpy(), want), name


# rows of one block, of each count of registers in both workgroup sizes, and
# of more than the registers hold
@pytest.mark.parametrize("q,cols", [(1, 32), (3, 96), (1, 4096), (4, 7168), (2, 4128), (5, 16384), (2, 32768), (2, 32800),
                                    (1, 131072), (600, 32), (513, 1056), (700, 2080), (520, 4128), (515, 8192), (514, 8224)])
@pytest.mark.parametrize("delta,weight", [(True, True), (False, False)])
def test_against_the_definition(q, cols, delta, weight):
    need_gpu()
    say(f"norm {q} x {cols} delta={delta} weight={weight}")
    x, d = rows(q, cols, q + cols), rows(q, cols, q + cols + 1) if delta else None
    w = 1 + 0.3 * rows(1, cols, 5, False)[0] if weight else None
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    o = outputs(q, cols)
    R.add_rms_norm(up(x), up(w), EPS, up(d), **o)
    check(o, *exact(x, d, w, EPS))
    # rfx_quantize_act's quotient and this product are half a step each from
    # max |y| / 127, and 1 / 127 another half
    xq, xs, xsum = (torch.empty_like(o[k]) for k in ("xq", "xs", "xsum"))
    R.quantize_act(o["y"], xq, xs, xsum)
    assert ((xs - o["xs"]).abs() <= xs * (3 * 2.0 ** -24 + 2.0 ** -40)).all()
    assert ((xq.int() - o["xq"].int()).abs() <= 1).all()
    # each output alone
    for names in (("out",), ("y",), ("xq", "xs", "xsum")):
        one = {k: v for k, v in outputs(q, cols).items() if k in names}
        R.add_rms_norm(up(x), up(w), EPS, up(d), **one)
        for k in names:
            assert torch.equal(one[k], o[k]), k


@pytest.mark.parametrize("q", [2, 600])
def test_strided_rows_and_aliases(q):
    need_gpu()
    cols = 1184
    wide, d = rows(q, cols + 96, 1).cuda(), rows(q, 3 * cols, 2).cuda()
    x, d = wide[:, 64:64 + cols], d[:, cols:2 * cols]
    h, y = exact(x.cpu(), d.cpu(), None, 1e-5)
    before = wide.clone()
    o = outputs(q, cols)
    R.add_rms_norm(x, None, 1e-5, d, **o)
    check(o, h, y)
    assert torch.equal(wide, before)
    # the stream updated in place, the norm over delta
    x, d = x.contiguous(), d.contiguous()
    R.add_rms_norm(x, None, 1e-5, d, out=x, y=d)
    assert torch.equal(x, o["out"]) and torch.equal(d, o["y"])
    # and where rows are read twice
    x, d = rows(2, 40000, 3), rows(2, 40000, 4)
    h, y = exact(x, d, None, 1e-5)
    x, d = x.cuda(), d.cuda()
    R.add_rms_norm(x, None, 1e-5, d, out=d, y=x)
    check(dict(out=d, y=x), h, y)


def test_rows_of_zeros_and_extremes():
    need_gpu()
    x = torch.zeros(6, 64)
    x[1, 5] = 1e-38
    x[2] = 3e38
    x[3] = -1e-45
    x[4, :32] = 1e-20
    x[5, 40] = 2.0
    for eps in (0.0, 1e-6):
        o = outputs(6, 64)
        R.add_rms_norm(x.cuda(), None, eps, **o)
        check(o, *exact(x, None, None, eps))
        assert not o["y"][0].any() and not o["xs"][0].any() and not o["xq"][0].any()


def test_no_rows():
    need_gpu()
    o = outputs(0, 64)
    R.add_rms_norm(torch.zeros(0, 64, device="cuda"), None, 1e-6, **o)


def test_captured_and_on_another_stream():
    torch = need_gpu()
    x, d = rows(3, 4096, 8).cuda(), rows(3, 4096, 9).cuda()
    o = outputs(3, 4096)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    R.add_rms_norm(x, None, EPS, d, **o, stream=s)
    s.synchronize()
    check(o, *exact(x.cpu(), d.cpu(), None, EPS))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.add_rms_norm(x, None, EPS, d, **o)
    for seed in (1, 2, 3):
        x.copy_(rows(3, 4096, seed))
        g.replay()
        torch.cuda.synchronize()
        check(o, *exact(x.cpu(), d.cpu(), None, EPS))


# both workgroup sizes, and rows that are read twice
@pytest.mark.parametrize("q,cols", [(7, 96), (7, 4128), (7, 32800), (520, 96), (520, 4128), (513, 8224)])
def test_what_is_not_finite(q, cols):
    """A row with a NaN is NaN in y and in every scale; one with an infinity
    is NaN there, in its block's scale, and zero elsewhere; an infinite or NaN
    weight stays in its column and block. Other rows are as they were."""
    need_gpu()
    say(f"norm {q} x {cols}, not finite")
    x, d = rows(q, cols, 1), rows(q, cols, 2)
    plain = outputs(q, cols)
    R.add_rms_norm(x.cuda(), None, EPS, d.cuda(), **plain)
    inf, nan = float("inf"), float("nan")
    places = {0: (cols - 1, nan, 1.0), 1: (5, 1.0, nan), 2: (40, inf, 1.0), 3: (cols - 20, -inf, 2.0), 4: (33, inf, -inf)}
    for r, (c, a, b) in places.items():
        x[r, c], d[r, c] = a, b
    o = outputs(q, cols)
    R.add_rms_norm(x.cuda(), None, EPS, d.cuda(), **o)
    h = (x + d).cuda()
    assert torch.equal(torch.isnan(o["out"]), torch.isnan(h)) and torch.equal(o["out"].nan_to_num(), h.nan_to_num())
    for r in (0, 1, 4): # inf - inf is NaN
        assert torch.isnan(o["y"][r]).all() and torch.isnan(o["xs"][r]).all()
    for r in (2, 3):
        c = places[r][0]
        there = torch.arange(cols, device="cuda") == c
        assert torch.equal(torch.isnan(o["y"][r]), there) and not o["y"][r][~there].any()
        block = torch.arange(cols // 32, device="cuda") == c // 32
        assert torch.equal(torch.isnan(o["xs"][r]), block) and not o["xs"][r][~block].any()
        assert not o["xq"][r].view(-1, 32)[~block].any() and not o["xsum"][r][~block].any()
    for k in o:
        assert torch.equal(o[k][5:], plain[k][5:]), k
    # codes alone say the same
    only = {k: v for k, v in outputs(q, cols).items() if k in ("xq", "xs", "xsum")}
    R.add_rms_norm(x.cuda(), None, EPS, d.cuda(), **only)
    for k in only:
        assert torch.equal(only[k].nan_to_num(), o[k].nan_to_num()) and torch.equal(torch.isnan(only[k]), torch.isnan(o[k])), k
    w = torch.ones(cols)
    w[7], w[70] = inf, nan
    o = outputs(q, cols)
    R.add_rms_norm(plain["out"], w.cuda(), EPS, **o)
    assert torch.isinf(o["y"][:, 7]).all() and torch.isnan(o["y"][:, 70]).all()
    assert torch.isinf(o["xs"][:, 0]).all() and torch.isnan(o["xs"][:, 2]).all()
    rest = [i for i in range(cols // 32) if i not in (0, 2)]
    assert torch.equal(o["xs"][:, rest], plain["xs"][:, rest]) and torch.equal(o["xsum"][:, rest], plain["xsum"][:, rest])


@pytest.mark.parametrize("fmt", ["FP2", "FP3", "FP4"])
@pytest.mark.parametrize("q", [1, 3, 7, 40])
def test_a_broken_row_shows_in_the_logits(q, fmt):
    need_gpu()
    g = torch.Generator().manual_seed(q)
    V, H = 320, 256
    head = R.DeviceHead.build(V, H, torch.randn(V, H, generator=g).numpy(), getattr(R, fmt), torch.ones(H).numpy())
    buf = R.HeadBuffers(head, q, 3)
    x = torch.randn(q, H, generator=g)
    want = buf.run(head, x.cuda()).lse.clone()
    assert torch.isfinite(want).all()
    for bad in (float("nan"), float("inf")):
        x[q - 1, 200] = bad
        p = buf.run(head, x.cuda())
        assert torch.equal(p.lse[:-1], want[:-1]) and torch.isnan(p.lse[-1]) and torch.isnan(p.entropy[-1])
