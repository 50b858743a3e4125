"""rfx_gemm against the oracle's dequantized weights in 64 bits: the GEMV form
(q <= 4, every format) and the matrix-core form, ragged rows and columns,
split K, every activation, residual in place, shared workspaces, graphs."""

import math

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R
import inputgen
import oracle as O
from gpu_common import need_gpu, quantize_on_gpu, say, upload_matrix

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def activate(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


class Case:
    def __init__(self, fmt, q, rows, cols, seed=0):
        self.fmt, self.q, self.rows, self.cols = fmt, q, rows, cols
        W = inputgen.dense_weight(rows, cols, seed=seed, outliers=True)
        x = inputgen.raw_normal(seed + 1, (q, cols))
        self.dW = upload_matrix(torch, fmt, W)
        self.xq, self.xs, self.xsum = quantize_on_gpu(torch, x)
        xd = self.xq.cpu().numpy().astype(np.float64) * np.repeat(self.xs.cpu().numpy().astype(np.float64), 32, axis=1)
        Wd = O.dequantize_matrix(fmt, O.quantize_matrix(fmt, W)).astype(np.float64)
        self.z, self.mag = xd @ Wd.T, np.abs(xd) @ np.abs(Wd).T
        self.bias = inputgen.raw_normal(seed + 2, (rows,), 0.3)
        self.resid = inputgen.raw_normal(seed + 3, (q, rows))

    def workspace(self):
        n = R.gemm_workspace_bytes(self.dW, self.q)
        return torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, act="none", bias=False, resid=False, ws=None, in_place=False, y=None):
        # y between two guards
        buf = torch.full((self.q * self.rows + 128,), 5.0, device="cuda")
        y = buf[64:64 + self.q * self.rows].view(self.q, self.rows)
        r = torch.from_numpy(self.resid).cuda() if resid else None
        if in_place:
            y.copy_(r)
            r = y
        R.gemm(self.dW, self.xq, self.xs, self.xsum, self.q, y, torch.from_numpy(self.bias).cuda() if bias else None,
               R.ACTIVATIONS[act], r, self.workspace() if ws is None else ws)
        torch.cuda.synchronize()
        assert (buf[:64] == 5).all() and (buf[64 + y.numel():] == 5).all(), "written outside y"
        return y.cpu().numpy().astype(np.float64)

    def check(self, y, act="none", bias=False, resid=False):
        """Each output is a sum over the cols / 32 blocks of an exact dot
        times a scale product that is rounded once: with one rounding per
        addition (any order) it is within (blocks + 2) 2^-24 of sum |w x|.
        Bias, activation (slope at most 1.13, its functions to a few 2^-24)
        and residual each round once."""
        z = self.z + (self.bias if bias else 0)
        want = activate(z, act) + (self.resid if resid else 0)
        tol = 1.13 * 2.0 ** -24 * ((self.cols // 32 + 2) * self.mag + np.abs(z)) + 2.0 ** -20 * np.abs(z) * (act != "none")
        tol += 2.0 ** -23 * (np.abs(want) + (np.abs(self.resid) if resid else 0)) + 1e-30
        bad = ~(np.abs(y - want) <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.abs(y - want)[bad].max()} at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("fmt", [2, 3, 4, 12, 8, 16, 13])
@pytest.mark.parametrize("q", [1, 2, 3, 4])
def test_few_columns(fmt, q):
    need_gpu()
    for i, (rows, cols) in enumerate(((1, 32), (100, 544), (320, 4096))):
        say(f"gemm fmt={fmt} q={q} {rows}x{cols}")
        c = Case(fmt, q, rows, cols, seed=10 * i + q)
        c.check(c.run(), "none")
        act = ACTS[(q + i) % 5]
        c.check(c.run(act, True, True), act, True, True)


@pytest.mark.parametrize("fmt", [2, 3, 4])
@pytest.mark.parametrize("q,rows,cols", [(5, 1, 32), (16, 64, 256), (17, 300, 800), (33, 257, 2080), (64, 130, 1056),
                                         (65, 200, 96), (129, 513, 544), (200, 90, 7168), (300, 1100, 320), (6, 5000, 512)])
def test_many_columns(fmt, q, rows, cols):
    need_gpu()
    say(f"gemm fmt={fmt} q={q} {rows}x{cols}")
    c = Case(fmt, q, rows, cols, seed=q)
    c.check(c.run())
    act = ACTS[q % 5]
    c.check(c.run(act, True, True), act, True, True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("q", [2, 40])
def test_activations_and_residual_in_place(act, q):
    need_gpu()
    c = Case(4, q, 200, 1024, seed=7)
    c.check(c.run(act), act)
    c.check(c.run(act, True), act, True)
    c.check(c.run(act, False, True, in_place=True), act, False, True)


def test_activation_tails():
    """Arguments far below and above zero: no NaN, and the tails themselves."""
    need_gpu()
    for q in (1, 20):
        c = Case(4, q, 64, 64, seed=3)
        c.bias = np.linspace(-3e4, 3e4, 64).astype(np.float32)
        c.bias[20:44] = np.linspace(-12, 12, 24)
        for act in ACTS:
            c.check(c.run(act, True), act, True)


def test_workspace_shared_by_all_forms():
    """One workspace through calls of few and many columns in turn: the
    GEMV form's exchange slots stay zero under the matrix-core form's data."""
    need_gpu()
    cases = [Case(3, 4, 1024, 2048, seed=1), Case(4, 100, 1024, 2048, seed=2), Case(2, 1, 200, 4096, seed=3),
             Case(4, 9, 300, 7168, seed=4)]
    n = max(R.gemm_workspace_bytes(c.dW, c.q) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    first = [c.run(ws=ws) for c in cases]
    for _ in range(2):
        for c, y in zip(cases, first):
            again = c.run(ws=ws)
            assert np.array_equal(again, y), "two runs differ"
            c.check(again)


@pytest.mark.parametrize("q", [3, 50])
def test_graph_replays(q):
    """Captured and replayed with the eager program's own calls between: every
    replay equals the eager result."""
    need_gpu()
    c = Case(4, q, 500, 4096, seed=5)
    bias, resid = torch.from_numpy(c.bias).cuda(), torch.from_numpy(c.resid).cuda()
    wg, we = c.workspace(), c.workspace()
    yg, ye = (torch.empty((q, 500), device="cuda") for _ in range(2))

    def call(y, ws):
        R.gemm(c.dW, c.xq, c.xs, c.xsum, q, y, bias, R.ACT_SILU, resid, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(yg, wg)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(yg, wg)
    for i in range(5):
        resid.mul_(1.5)
        c.xs.mul_(0.75)
        call(ye, we)
        torch.cuda.synchronize()
        yg.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, ye), i


def wide_case(q, rows, cols, seed):
    """FP4 weights and activations whose block scales are far apart, codes of
    every size (a block's largest from 1 to -128) and zero blocks."""
    rng = np.random.default_rng(seed)
    nb = cols // 32
    c = Case(4, q, rows, cols, seed=seed)
    W = inputgen.dense_weight(rows, cols, seed=seed) * np.repeat(2.0 ** rng.integers(-12, 13, (rows, nb)), 32, axis=1)
    W = W.astype(np.float32)
    c.dW = upload_matrix(torch, 4, W)
    c.Wd = O.dequantize_matrix(4, O.quantize_matrix(4, W)).astype(np.float64)
    amp = 2.0 ** rng.uniform(0, 7, (q, nb))
    amp[rng.random((q, nb)) < 0.1] = 0
    codes = np.round(rng.uniform(-1, 1, (q, nb, 32)) * amp[..., None])
    codes[0, 0, 5] = -128
    xs = (2.0 ** rng.uniform(-20, 20, (q, nb))).astype(np.float32)
    xs[rng.random((q, nb)) < 0.05] = 0
    if q > 1 and nb > 1:
        xs[1, 1] = 1e-41  # subnormal
    return c, codes.astype(np.int8), xs


@pytest.mark.parametrize("q,rows,cols", [(5, 70, 32), (9, 100, 512), (40, 300, 800), (130, 600, 2080)])
def test_fp4_digits_over_wide_scales(q, rows, cols):
    """FP4's activations as sums of five digits: each is within 2^-23.9 of the
    largest of its block after the fp32 rounding of code * scale (2^-24), the
    ten products of a K tile round once each at no more than the tile's sum of
    |w x|, and each of the tiles is added with one rounding: within
    (tiles + 11) 2^-24 sum |w x| + 2^-23.9 sum_b max_b |x| sum_b |w|. Partials
    of up to tiles / 2 splits add as many roundings."""
    need_gpu()
    say(f"gemm wide q={q} {rows}x{cols}")
    c, codes, xs = wide_case(q, rows, cols, seed=q)
    nb = cols // 32
    c.xq = torch.from_numpy(codes.reshape(q, cols)).cuda()
    c.xs = torch.from_numpy(xs).cuda()
    c.xsum = torch.from_numpy(codes.astype(np.int32).sum(2).astype(np.int32)).cuda()
    y = c.run()
    xd = codes.astype(np.float64) * xs[..., None].astype(np.float64)
    want = xd.reshape(q, cols) @ c.Wd.T
    mag = np.abs(xd).reshape(q, cols) @ np.abs(c.Wd).T
    top = np.abs(xd).max(2) @ np.abs(c.Wd).reshape(rows, nb, 32).sum(2).T
    tiles = -(-cols // 256)
    tol = 2.0 ** -24 * (1.5 * tiles + 11) * mag + 2.0 ** -23.9 * top + 1e-30
    bad = ~(np.abs(y - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {(np.abs(y - want) / tol)[bad].max()} of its bound"


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_fp4_scale_that_is_not_finite(value):
    """A block whose largest value is not finite (3e38 * 127 neither) makes
    its column NaN and no other."""
    need_gpu()
    c = Case(4, 20, 100, 512, seed=2)
    c.xs[3, 4] = value
    y = c.run()
    assert np.isnan(y[3]).all() and np.isfinite(np.delete(y, 3, 0)).all()
    keep = [j for j in range(20) if j != 3]
    tol = 1.13 * 2.0 ** -24 * (512 // 32 + 2) * c.mag + 1e-30
    assert (np.abs(y - c.z) <= tol)[keep].all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("q", [2, 40])
def test_nan_reaches_the_result(act, q):
    """A NaN before the activation is one after it, in its row only."""
    need_gpu()
    c = Case(4, q, 70, 512, seed=4)
    c.bias[9] = np.nan
    y = c.run(act, True)
    assert np.isnan(y[:, 9]).all() and np.isfinite(np.delete(y, 9, 1)).all()


@pytest.mark.parametrize("fmt", [2, 3, 4])
@pytest.mark.parametrize("q,rows,cols", [(30, 2900, 4192), (64, 2100, 5600), (100, 1300, 4128), (260, 1100, 3200),
                                         (1400, 4100, 64)])
def test_many_columns_that_fill_the_device(fmt, q, rows, cols):
    """Sizes at which workgroups take 32 to 128 columns (smaller matrices
    take fewer per workgroup), and FP4's 512 rows."""
    need_gpu()
    say(f"gemm fmt={fmt} q={q} {rows}x{cols}")
    c = Case(fmt, q, rows, cols, seed=q)
    c.check(c.run())
    act = ACTS[q % 5]
    c.check(c.run(act, True, True), act, True, True)


@pytest.mark.parametrize("rows,cols", [(2560, 8192), (5632, 4096), (3008, 8192)])
def test_workspace_shared_where_slots_are_many(rows, cols):
    """The same where the GEMV form's exchange slots take the most: a call of
    64 columns writes its operands behind them."""
    need_gpu()
    few, many = Case(4, 4, rows, cols, seed=1), Case(4, 64, rows, cols, seed=2)
    ws = torch.zeros(max(R.gemm_workspace_bytes(c.dW, c.q) for c in (few, many)), dtype=torch.uint8, device="cuda")
    first = few.run(ws=ws)
    few.check(first)
    for _ in range(2):
        many.check(many.run(ws=ws))
        assert np.array_equal(few.run(ws=ws), first)


@pytest.mark.parametrize("fmt", [3, 4])
@pytest.mark.parametrize("q", [2, 40])
def test_unaligned_results_and_residuals(fmt, q):
    """y, resid and bias at 4-byte addresses, with rows a multiple of four."""
    need_gpu()
    c = Case(fmt, q, 512, 544, seed=6)
    bufs = [torch.full((q * 512 + 8,), 5.0, device="cuda") for _ in range(2)]
    for at, ar in ((1, 0), (0, 3), (2, 1)):
        y, r = (b[4 + o:4 + o + q * 512].view(q, 512) for b, o in zip(bufs, (at, ar)))
        bufs[0].fill_(5.0)
        r.copy_(torch.from_numpy(c.resid))
        bias = torch.zeros(513, device="cuda")
        bias[1:] = torch.from_numpy(c.bias)
        R.gemm(c.dW, c.xq, c.xs, c.xsum, q, y, bias[1:], R.ACT_GELU, r, c.workspace())
        c.check(y.cpu().numpy().astype(np.float64), "gelu", True, True)
        assert (bufs[0][:4 + at] == 5).all() and (bufs[0][4 + at + q * 512:] == 5).all()


@pytest.mark.parametrize("q", [4, 40])
def test_buffers_larger_than_the_call(q):
    """The first q columns of larger activation buffers."""
    need_gpu()
    c = Case(4, q + 9, 200, 1024, seed=6)
    y = torch.full((q + 9, 200), 5.0, device="cuda")
    n = R.gemm_workspace_bytes(c.dW, q)
    R.gemm(c.dW, c.xq, c.xs, c.xsum, q, y, ws=torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None)
    assert (y[q:] == 5).all()
    c.z, c.mag = c.z[:q], c.mag[:q]
    c.check(y[:q].cpu().numpy().astype(np.float64))
