"""rfx_token_logprobs against its definition in 64 bits: sums, entropies,
ranks, and the largest logits with ties to the lower index; excluded tokens,
rows that nothing is left of, rows whose order is the worst for the selection."""

import math

import pytest
import torch

import bit_block_quantized_amd as R
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def exact(z, tokens, k):
    """In 64 bits, with bounds on the kernel's error. An exponential's
    argument d = z - m is rounded once and times log2 e once (|d| steps of
    2^-24 each), the hardware's exp2 is good to 2^-23; a thread adds up to 32
    of them, a wave and the four waves 9 more, chunks are added in 64 bits: a
    relative error of s of (2 |d| + 2 + 41 + 3) 2^-24 on average over p. The
    entropy's sum has the same per term, of p |d| each."""
    z = z.double()
    m = z.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    d = z - m0
    e = d.exp()
    s = e.sum(-1, keepdim=True)
    p = e / torch.where(s == 0, 1.0, s)
    dz = torch.where(e > 0, d, 0.0)
    D, D2 = (p * dz.abs()).sum(-1), (p * dz * dz).sum(-1)
    step = 2.0 ** -24
    # log s without the largest's 1, which a small rest would be lost behind
    # (64 bits lose it from 2^-53 on)
    first = torch.zeros_like(e).scatter_(1, z.argmax(-1, keepdim=True), 1.0)
    ls = torch.where(s[:, 0] > 0, torch.where(first > 0, 0.0, e).sum(-1), 0.0).log1p()
    lse = torch.where(s[:, 0] > 0, m0[:, 0] + ls, -math.inf)
    t_s = (2 * D + 50) * step * -torch.expm1(-ls) # the count of the largest is exact
    r = dict(lse=(lse, t_s + step * lse.abs()), entropy=(ls - (p * dz).sum(-1), t_s * (1 + D) + (2 * D2 + 50 * D) * step))
    r["entropy"] = (r["entropy"][0], r["entropy"][1] + step * r["entropy"][0].abs() + 2.0 ** -100)
    known = (tokens >= 0) & (tokens < z.shape[1])
    zt = z.gather(1, tokens.clamp(0, z.shape[1] - 1).long()[:, None])
    # in 64 bits from the chunks' sums on, one rounding
    lp = torch.where(known, torch.where(zt[:, 0] == -math.inf, -math.inf, zt[:, 0] - m0[:, 0] - ls), 0.0)
    r["logprob"] = (lp, t_s + step * lp.abs() + 2.0 ** -100)
    r["rank"] = torch.where(known, (z > zt).sum(-1), -1)
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :k]
    best = z.gather(1, order)
    gone = best == -math.inf
    n = order.shape[1]
    top = torch.full((z.shape[0], k), -1)
    top[:, :n] = torch.where(gone, -1, order)
    tl = torch.full((z.shape[0], k), -math.inf, dtype=torch.float64)
    tl[:, :n] = torch.where(gone, -math.inf, best - m0 - ls[:, None])
    r["top_index"], r["top_logprob"] = top, (tl, t_s[:, None] + step * tl.abs() + 2.0 ** -100)
    return r


def check(z, tokens, k, buf=None):
    """z: CPU tensor of logits, rows may be strided."""
    need_gpu()
    q, V = z.shape
    say(f"logprobs {q} x {V} {z.dtype} stride {z.stride(0)} k={k}")
    zd = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda")
    zd.copy_(z)
    buf = buf or R.LogprobBuffers(q, V, k)
    buf.ws.fill_(255)
    for t in (buf.logprob, buf.lse, buf.entropy, buf.top_logprob):
        t.fill_(7.0)
    buf.run(zd, tokens.to(torch.int32).cuda())
    ref = exact(z, tokens, k)
    names = ["lse", "entropy", "logprob"] + ["top_logprob"] * (k > 0)
    for name in names:
        want, tol = ref[name]
        got = getattr(buf, name).cpu().double()
        same = got == want # infinities among them
        bad = ~(same | ((got - want).abs() <= tol))
        assert not bad.any(), f"{name}: {got[bad][:3]} {want[bad][:3]}"
    assert torch.equal(buf.rank.cpu().long(), ref["rank"])
    if k:
        assert torch.equal(buf.top_index.cpu().long(), ref["top_index"]), "order"
    return buf


def logits(q, V, seed, kind="f32", sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(q, V, generator=g) * sigma).to(TYPES[kind]), torch.randint(0, V, (q,), generator=g)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("q,V,k", [(1, 1, 1), (2, 2, 5), (1, 7, 0), (3, 63, 64), (2, 500, 20), (1, 2048, 5), (2, 2049, 64),
                                   (3, 8185, 3), (1, 8192, 64), (2, 20001, 8), (1, 100003, 64), (70, 8193, 20), (600, 777, 4),
                                   (40, 131072, 10), (1, 1 << 19, 64)])
def test_sizes(q, V, k, kind):
    z, t = logits(q, V, q + V + k, kind)
    check(z, t, k)


@pytest.mark.parametrize("kind", list(TYPES))
def test_rows_at_any_address(kind):
    """Rows that start anywhere in 16 bytes, of a tensor that itself does,
    with NaN around them."""
    need_gpu()
    q, V, k = 9, 4099, 12
    z, t = logits(q, V, 3, kind)
    for stride in (4099, 4100, 4107, 4200):
        for first in range(0, 9, 1 if stride == 4099 else 4):
            flat = torch.full((first + q * stride,), float("nan"), dtype=z.dtype)
            view = flat[first:].as_strided((q, V), (stride, 1))
            view.copy_(z)
            fd = flat.cuda()
            zd = fd[first:].as_strided((q, V), (stride, 1))
            b = R.LogprobBuffers(q, V, k).run(zd, t.to(torch.int32).cuda())
            ref = exact(z, t, k)
            assert torch.equal(b.top_index.cpu().long(), ref["top_index"]) and torch.equal(b.rank.cpu().long(), ref["rank"])
            for name in ("lse", "entropy", "logprob", "top_logprob"):
                want, tol = ref[name]
                assert ((getattr(b, name).cpu().double() - want).abs() <= tol).all(), name


# what the selection's bound meets at its worst: equal logits, ascending and
# descending ones, the largest side by side, all in one thread's places
def _orders(V):
    i = torch.arange(V, dtype=torch.float32)
    return {"equal": torch.zeros(V), "signed zeros": torch.where(i % 2 == 0, 0.0, -0.0), "ascending": i / V * 20,
            "descending": -i / V * 20, "side by side": torch.where((i > V // 3) & (i < V // 3 + 300), 9.0 + i / V, -i / V),
            "one thread": torch.where(i % 1024 < 4, 5.0 + (i % 7), 0.0), "two values": (i % 3 == 1).float(),
            "one likely": torch.where(i == V // 2, 25.0, 0.0), "very likely": torch.where(i == V - 1, 40.0, -i / V)}


@pytest.mark.parametrize("V", [300, 5000, 40000])
@pytest.mark.parametrize("k", [1, 20, 64])
def test_orders(V, k):
    rows = _orders(V)
    z = torch.stack(list(rows.values()))
    check(z, torch.arange(len(rows)) * 17 % V, k)


def test_the_small_rest_is_kept():
    """One token of probability 1 - 1e-9: its log probability and the row's
    entropy are far below an fp32 step of 1."""
    z = torch.full((2, 1000), -30.0)
    z[0, 500], z[1, 3] = 0.0, 0.0
    z[1, 4] = -22.0
    b = check(z, torch.tensor([500, 3]), 2)
    assert -1.1e-10 * 999 < float(b.logprob[0]) < -0.9e-13 * 999 and 0 < float(b.entropy[0]) < 1e-8


def test_excluded_tokens():
    need_gpu()
    V, inf = 9000, math.inf
    g = torch.Generator().manual_seed(4)
    z = torch.randn(7, V, generator=g)
    z[0] = -inf                      # nothing is left
    z[1, 5:] = -inf                  # five are
    z[2, :8500] = -inf               # whole chunks are excluded
    z[3, torch.arange(V) % 2 == 0] = -inf
    z[4] = torch.finfo(torch.float32).min # the type's lowest value is a logit like any other
    z[5, :8200] = torch.finfo(torch.float32).min
    z[6] = -inf
    z[6, 8999] = -3e38               # one is left, far down
    b = check(z, torch.tensor([3, 6, 8600, 1, 2, 8300, 8999]), 20)
    assert float(b.entropy[0]) == 0 and float(b.lse[0]) == -inf and float(b.logprob[0]) == -inf
    assert float(b.logprob[1]) == -inf and float(b.logprob[6]) == 0
    assert (b.top_index[0] == -1).all() and (b.top_index[1, 5:] == -1).all() and (b.top_logprob[1, 5:] == -inf).all()


def test_tokens_that_are_none():
    z, _ = logits(4, 333, 9)
    t = torch.tensor([-1, 333, 2 ** 31 - 1, 0])
    b = check(z, t, 3)
    assert b.rank.tolist()[:3] == [-1, -1, -1] and b.logprob.tolist()[:3] == [0, 0, 0]
    # without tokens logprob and rank stay
    b.logprob.fill_(7.0)
    b.rank.fill_(7)
    b.run(z.cuda())
    assert (b.logprob == 7).all() and (b.rank == 7).all()


def test_what_is_not_finite():
    need_gpu()
    z, t = logits(4, 9000, 10)
    ref = exact(z[3:], t[3:], 5)
    z[0, 7], z[1, 8990], z[2, 10] = math.nan, math.inf, math.nan
    z[2, 11:] = -math.inf
    b = R.LogprobBuffers(4, 9000, 5).run(z.cuda(), t.to(torch.int32).cuda())
    assert torch.isnan(b.lse[:3]).all() and torch.isnan(b.entropy[:3]).all() and torch.isnan(b.logprob[:3]).all()
    assert torch.equal(b.top_index[3:].cpu().long(), ref["top_index"])
    assert int(b.top_index[1, 0]) == 8990 and ((b.top_index >= -1) & (b.top_index < 9000)).all()


def test_captured_and_deterministic():
    torch = need_gpu()
    z, t = logits(5, 30000, 11)
    zd, td = z.cuda(), t.to(torch.int32).cuda()
    b = R.LogprobBuffers(5, 30000, 7)
    b.run(zd, td)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(zd, td)
    for seed in (12, 13, 12):
        z, t = logits(5, 30000, seed)
        zd.copy_(z)
        td.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        ref = exact(z, t, 7)
        assert torch.equal(b.top_index.cpu().long(), ref["top_index"])
        assert ((b.lse.cpu().double() - ref["lse"][0]).abs() <= ref["lse"][1]).all()
        again = R.LogprobBuffers(5, 30000, 7).run(zd, td)
        for name in ("logprob", "lse", "entropy", "rank", "top_index", "top_logprob"):
            assert torch.equal(getattr(again, name), getattr(b, name)), name


@pytest.mark.parametrize("kind", list(TYPES))
def test_borders_of_long_chunks(kind):
    """Rows that end beside the end of a chunk, so many that chunks are long
    ones, with few alternatives and with more."""
    n = 1536 * (1 if kind == "f32" else 2) # of one wave, of four: four times that
    for q, V, k in ((1100, n - 3, 5), (1100, n + 1, 1), (300, 4 * n - 3, 20), (300, 4 * n + 1, 64)):
        check(*logits(q, V, V + k, kind), k)
    for q, V, k in ((1100, n + 1, 8), (300, 4 * n + 1, 20)):
        z = torch.stack(list(_orders(V).values())).repeat(q // 9 + 1, 1)[:q].to(TYPES[kind])
        check(z, torch.arange(q) % V, k)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [0, 5, 20])
@pytest.mark.parametrize("q", [9, 600])
def test_finite_values_of_any_size(q, k, kind):
    """Tokens excluded by a large finite number, or rows that are nothing
    else: whole waves and chunks of them beside ordinary logits, in short
    chunks and long ones."""
    V = 5000
    g = torch.Generator().manual_seed(q + k)
    i = torch.arange(V)
    per = 256 if kind == "f32" else 512 # what a wave takes at a time
    masks = [i < 2048 if kind == "f32" else i < 4096, i >= 3000, i % (4 * per) < per, i % (4 * per) >= per, i >= 0, i != 77]
    rows = []
    for value in (1e4, 1e7, 1e9, 3e9, 1e10, 3e10, 1e13, 1e20, 1e30, 1e38, 2e38, 3.3e38):
        for sign in (-1.0, 1.0):
            for j, m in enumerate(masks):
                z = torch.randn(V, generator=g) * 3
                # the same number everywhere, or near it (some steps of fp32 below)
                rows.append(torch.where(m, sign * value * (1 if j % 2 else 1 - (i % 5) * 2.0 ** -22), z))
    z = torch.stack(rows).to(TYPES[kind])
    t = torch.randint(0, V, (len(z),), generator=g)
    for at in range(0, len(z), q):
        part = torch.arange(at, at + q) % len(z)
        check(z[part], t[part], k)
