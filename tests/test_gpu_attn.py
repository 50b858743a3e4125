"""rfx_attn against its definition in 64 bits: decode (few rows per kv
head), split and joined keys, prompts, windows with sinks, pages that end
inside tiles, bad page ids, rows of no sequence, captured graphs."""

import pytest
import torch

import bit_block_quantized_amd as R
from attn_common import TYPES, Batch, attn_bound, attn_exact
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


def run(b, q, scale, window=0, sinks=0, out="f32", ws=None):
    cache, batch = b.device(R)
    heads = q.shape[1]
    dtype = torch.float32 if out == "f32" else b.dtype
    o = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    n = R.attn_workspace_bytes(cache, batch, heads)
    if ws is None and n:
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN: it needs no initialisation
    R.attn(q.cuda(), cache, batch, o, scale, window, sinks, ws)
    torch.cuda.synchronize()
    return o.cpu()


def check(lens, heads, kv_heads, dim, page, kind, window=0, sinks=0, out="f32", scale=None, seed=0, **kw):
    need_gpu()
    say(f"attn {lens[:4]} h={heads}/{kv_heads} d={dim} page={page} {kind} w={window}+{sinks} -> {out}")
    b = Batch(lens, page, kv_heads, dim, kind, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((b.n_tokens, heads, dim), generator=g).to(TYPES[kind])
    scale = dim ** -0.5 if scale is None else scale
    o = run(b, q, scale, window, sinks, out)
    ref, mag, dots = attn_exact(b, q, scale, window, sinks)
    rows = b.max_q * (heads // kv_heads)
    tol = attn_bound(b, ref, mag, dots, o.dtype, out != "f32" and rows > 16)
    idle = torch.isnan(ref)
    assert torch.equal(o.double()[idle], torch.full_like(ref, 7.0)[idle]), "rows of no sequence were written"
    bad = ~((o.double() - ref).abs() <= tol) & ~idle
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside: {(o.double() - ref).abs()[bad].max()} at {bad.nonzero()[0].tolist()}"
    return b, q, o


# (lens, heads, kv_heads, dim, page): one token to a few hundred, odd group
# sizes, every head-dim class, pages from one token to more than a sequence
DECODE = [
    ([(1, 1)], 4, 4, 64, 16),
    ([(1, 37)], 8, 2, 128, 16),
    ([(1, 300)], 6, 2, 128, 32),
    ([(4, 259), (4, 4), (4, 33)], 8, 1, 128, 64),
    ([(2, 130), (0, 50), (3, 3), (1, 0), (4, 511)], 16, 4, 64, 1),
    ([(3, 700), (1, 65)], 5, 1, 80, 8),
    ([(1, 1025), (1, 31), (1, 32)], 16, 1, 256, 32),
    ([(4, 100)], 4, 1, 200, 4),
    ([(2, 90), (2, 64)], 2, 2, 8, 256),
    ([(1, 77)] * 9, 20, 4, 120, 2),
    ([(2, 300), (1, 50)], 8, 2, 256, 16),
    ([(1, 2500), (4, 1000)], 8, 2, 128, 16),
    ([(1, 9000)], 2, 1, 64, 128),
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, kind):
    lens, heads, kv, dim, page = DECODE[case]
    check(lens, heads, kv, dim, page, kind, seed=case, lead=case % 2, tail=case % 3)
    check(lens, heads, kv, dim, page, kind, out="same", seed=100 + case)


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (40, 4), (64, 33), (100, 500), (2000, 4)])
def test_decode_window(window, sinks, page):
    check([(4, 333), (1, 40), (2, 1200)], 8, 2, 64, page, "bf16", window, sinks)


def test_decode_split_and_joined():
    """One sequence, one kv head: the keys are split over workgroups."""
    for kind, page, total in (("f16", 64, 9000), ("bf16", 16, 5003), ("bf16", 256, 4097)):
        b, q, o = check([(1, total)], 8, 1, 128, page, kind, seed=total)
        assert R.attn_workspace_bytes(b.cache, b.batch, 8) > 0
        again = run(b, q, 128 ** -0.5)
        assert torch.equal(again, o), "two runs differ"


PROMPT = [
    ([(5, 5)], 16, 2, 64, 16),
    ([(33, 33)], 4, 2, 128, 16),
    ([(130, 130)], 3, 1, 128, 32),
    ([(64, 200), (0, 9), (1, 1), (17, 300), (129, 129)], 8, 2, 64, 8),
    ([(40, 333)], 5, 1, 80, 1),
    ([(70, 70), (9, 140)], 4, 2, 256, 64),
    ([(50, 90)], 2, 2, 24, 4),
    ([(1, 700), (4, 65)], 48, 1, 128, 16),
    ([(4, 300)], 16, 2, 256, 32),
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "same"])
@pytest.mark.parametrize("case", range(len(PROMPT)))
def test_prompt(case, kind, out):
    lens, heads, kv, dim, page = PROMPT[case]
    check(lens, heads, kv, dim, page, kind, out=out, seed=200 + case, lead=case % 3, tail=case % 2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (30, 4), (64, 65), (129, 500), (5000, 1)])
def test_prompt_window(window, sinks, dim):
    check([(200, 200), (40, 400), (6, 6)], 4, 2, dim, 16, "bf16", window, sinks, out="f32")
    check([(77, 500)], 4, 1, dim, 64, "f16", window, sinks, out="same")


def test_prompt_split_and_joined():
    """A short chunk late in a long sequence: few row blocks, split keys."""
    for kind, out in (("bf16", "same"), ("f16", "f32")):
        b, q, o = check([(40, 6000)], 8, 1, 128, 32, kind, out=out, seed=5)
        assert R.attn_workspace_bytes(b.cache, b.batch, 8) > 0
        assert torch.equal(run(b, q, 128 ** -0.5, out=out), o), "two runs differ"


def test_large_scores_and_far_keys():
    """Scores of hundreds (one key takes nearly all weight; later tiles raise
    the maximum) and a scale far from 1 / sqrt(dim)."""
    for rows in (1, 60):
        check([(rows, 900)], 8, 2, 64, 16, "f16", scale=4.0, seed=9)
        check([(rows, 900)], 8, 2, 64, 16, "bf16", scale=1e-3, seed=9)


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("page", [4, 64])
def test_rows_before_the_first_token(rows, page):
    """kv_len below the number of new tokens: the first rows are at negative
    positions, see nothing and are zero."""
    check([(rows, rows - 1), (rows, 0)], 8, 2, 64, page, "bf16", window=0, seed=3)


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("page", [2, 16, 32])
def test_bad_pages_are_not_visible(rows, page):
    """A page id outside the cache: its keys count as masked; a sequence with
    no good page is zero."""
    need_gpu()
    b = Batch([(rows, 200), (rows, 150)], page, 2, 64, "bf16", seed=4)
    for j in range(0, b.table.shape[1], 3):
        b.table[0, j] = (-1, b.n_pages, 1 << 30)[j % 3]
    b.table[1, :] = -5
    q = torch.randn((2 * rows, 4, 64), generator=torch.Generator().manual_seed(6)).to(b.dtype)
    o = run(b, q, 0.125)
    good = (b.table >= 0) & (b.table < b.n_pages)
    # the definition over the keys whose pages are good
    for h in range(4):
        for i in range(rows):
            keys = [p for p in range(200 - rows + i + 1) if good[0, p // page]]
            k = torch.stack([b.k[int(b.table[0, p // page]), h // 2, p % page] for p in keys]).double()
            v = torch.stack([b.v[int(b.table[0, p // page]), h // 2, p % page] for p in keys]).double()
            w = torch.softmax(k @ q[i, h].double() * 0.125, 0)
            # weights to 2^-16 (scores below 10, 64 products, 200 keys: see attn_bound)
            assert ((o[i, h].double() - w @ v).abs() <= 2.0 ** -16 * (w @ v.abs())).all(), (i, h)
    assert not o[rows:].any()


@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("page", [4, 16, 64])
def test_masked_nan_stays_out(rows, page):
    """NaN and infinity in keys and values that every row's window leaves
    out, beside the visible ones of the same page and tile."""
    need_gpu()
    b = Batch([(rows, 333)], page, 1, 64, "f16", seed=8)
    lo = 333 - rows - 20 + 1
    for p in range(3, lo):
        at = int(b.table[0, p // page]), slice(None), p % page
        b.k[at] = float("nan") if p % 2 else float("inf")
        b.v[at] = float("-inf") if p % 2 else float("nan")
    q = torch.randn((rows, 4, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    o = run(b, q, 0.125, window=20, sinks=3)
    ref, mag, dots = attn_exact(b, q, 0.125, 20, 3)
    assert ((o.double() - ref).abs() <= attn_bound(b, ref, mag, dots, o.dtype, False)).all()


def test_rows_past_max_q_and_past_the_arrays():
    """Rows past max_q are left, and a sequence whose rows leave the arrays
    is skipped."""
    need_gpu()
    b = Batch([(3, 40), (9, 60)], 16, 2, 64, "bf16", seed=11, max_q=3)
    q = torch.randn((12, 4, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    o = run(b, q, 0.125)
    ref, mag, dots = attn_exact(b, q, 0.125)
    ok = (o.double() - ref).abs() <= attn_bound(b, ref, mag, dots, o.dtype, False)
    assert ok[:6].all() and (o[6:] == 7).all()
    b.q_off[2] = 13
    o = run(b, q, 0.125)
    assert ((o.double() - ref).abs() <= attn_bound(b, ref, mag, dots, o.dtype, False))[:3].all() and (o[3:] == 7).all()


@pytest.mark.parametrize("lens,heads", [([(1, 3000), (1, 2000)], 4), ([(40, 3000)], 8)])
def test_graph_replays_with_growing_sequences(lens, heads):
    """A captured call replayed with the eager program's own calls between,
    the device arrays changed for each replay: every replay equals the eager
    result."""
    need_gpu()
    b = Batch(lens, 32, 1, 64, "bf16", seed=12)
    q = torch.randn((b.n_tokens, heads, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype).cuda()
    cache, batch = b.device(R)
    n = R.attn_workspace_bytes(cache, batch, heads)
    assert n > 0
    wg, we = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    og, oe = (torch.empty(q.shape, dtype=torch.float32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.attn(q, cache, batch, og, 0.125, 0, 0, wg)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        R.attn(q, cache, batch, og, 0.125, 0, 0, wg)
    for i in range(5):
        batch.kv_len.copy_((b.kv_len.cuda() - 211 * i).to(torch.int32))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(20 + i)).to(b.dtype))
        R.attn(q, cache, batch, oe, 0.125, 0, 0, we)
        torch.cuda.synchronize()
        og.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, oe), i


def test_other_stream():
    need_gpu()
    b = Batch([(1, 800), (1, 90)], 16, 2, 64, "f16", seed=13)
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    want = run(b, q, 0.125)
    cache, batch = b.device(R)
    qd, o = q.cuda(), torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    ws = torch.zeros(max(1, R.attn_workspace_bytes(cache, batch, 8)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    R.attn(qd, cache, batch, o, 0.125, 0, 0, ws, stream=s)
    s.synchronize()
    assert torch.equal(o.cpu(), want)


def test_cache_past_32_bit_offsets():
    """A cache of more than 2^32 bytes of keys, the sequence's pages at its
    end: offsets need more than 32 bits."""
    need_gpu()
    pages, page, kv, dim = 36000, 64, 8, 128  # 2.36 G elements, 4.7 GB each of keys and values
    b = Batch([(1, 200), (40, 130)], page, kv, dim, "bf16", seed=14)
    b.n_pages = pages
    big = [torch.zeros((pages, kv, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = pages - b.k.shape[0]
    big[0][shift:], big[1][shift:] = b.k.cuda(), b.v.cuda()
    small = b.table.clone()
    ok = (small >= 0) & (small < b.k.shape[0])
    table = torch.where(ok, small + shift, small)
    cache = R.DeviceKVCache(*big)
    q = torch.randn((41, 16, dim), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    ref, mag, dots = attn_exact(b, q, 0.1)
    tol = attn_bound(b, ref, mag, dots, torch.float32, False)
    for lo, hi, seqs, mq in ((0, 1, slice(0, 1), 1), (1, 41, slice(1, 2), 40)):
        off = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        batch = R.KVBatch(off, b.kv_len[seqs].cuda(), table[seqs].cuda().contiguous(), hi - lo, mq)
        o = torch.empty((hi - lo, 16, dim), dtype=torch.float32, device="cuda")
        n = R.attn_workspace_bytes(cache, batch, 16)
        R.attn(q[lo:hi].cuda(), cache, batch, o, 0.1, 0, 0, torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda"))
        assert ((o.cpu().double() - ref[lo:hi]).abs() <= tol[lo:hi]).all()


# Calls of 512 and more blocks of 256 rows, heads over 64: the kernel of two
# wave groups. Rows over blocks, groups and waves
# that are full, partial and empty; pages from one token to 128.
MANY = [
    ([(40, 40)] * 61 + [(300, 300), (0, 70), (33, 500)], 8, 8, 128, 16, 0, 0),
    ([(33, 33 + 7 * i) for i in range(64)], 8, 8, 72, 64, 0, 0),
    ([(35, 100 + 3 * i) for i in range(64)], 8, 8, 128, 1, 50, 3),
    ([(70, 70 + i) for i in range(66)], 16, 8, 96, 32, 30, 0),
    ([(200, 200), (1, 600), (257, 400), (64, 64)] + [(40, 300)] * 252, 2, 2, 128, 128, 129, 70),
]
# The same with split keys: tables of a capacity (more entries than needed)
# that makes long runs.
MANY_SPLIT = [
    ([(40, 600)] * 32, 8, 8, 128, 64, 0, 0, 130),
    ([(33, 900 - 9 * i) for i in range(64)], 4, 4, 80, 32, 0, 2, 260),
    ([(70, 2000), (300, 1500)], 8, 4, 128, 128, 700, 90, 680),
]


@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("bf16", "f32"), ("f16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_two_groups(case, kind, out):
    lens, heads, kv, dim, page, window, sinks = MANY[case]
    check(lens, heads, kv, dim, page, kind, window, sinks, out=out, seed=300 + case, lead=case % 2, tail=case % 3)


@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("case", range(len(MANY_SPLIT)))
def test_two_groups_split_and_joined(case, kind, out):
    lens, heads, kv, dim, page, window, sinks, more = MANY_SPLIT[case]
    b, q, o = check(lens, heads, kv, dim, page, kind, window, sinks, out=out, seed=400 + case, extra_entries=more)
    assert R.attn_workspace_bytes(b.cache, b.batch, heads) > 0
    assert torch.equal(run(b, q, dim ** -0.5, window, sinks, out), o), "two runs differ"


@pytest.mark.parametrize("page", [2, 16, 64, 128])
def test_two_groups_bad_pages_and_nan(page):
    """Bad page ids mask their keys, and what no row sees may be NaN, where
    blocks of both groups are at work; two runs agree."""
    need_gpu()
    b = Batch([(34, 234)] * 64, page, 8, 128, "bf16", seed=21)
    stride = b.table.shape[1]
    for s in range(64):
        for j in range(s % 3, stride, 3 + s % 2):
            b.table[s, j] = (-1, b.n_pages, 1 << 30)[j % 3]
    q = torch.randn((34 * 64, 8, 128), generator=torch.Generator().manual_seed(6)).to(b.dtype)
    o = run(b, q, 0.1, window=60, sinks=5)
    assert torch.equal(o, run(b, q, 0.1, window=60, sinks=5))
    for s in range(0, 64, 7):
        good = [(int(b.table[s, p // page]), p % page) if 0 <= int(b.table[s, p // page]) < b.n_pages else None for p in range(234)]
        for i in (0, 15, 33):
            pos = 200 + i
            keys = [good[p] for p in range(pos + 1) if good[p] and (p > pos - 60 or p < 5)]
            for h in (0, 7):
                if not keys:
                    assert not o[34 * s + i, h].any()
                    continue
                k = torch.stack([b.k[a, h, c] for a, c in keys]).double()
                v = torch.stack([b.v[a, h, c] for a, c in keys]).double()
                w = torch.softmax(k @ q[34 * s + i, h].double() * 0.1, 0)
                # weights to 2^-15 (scores below 10, 128 products, 65 keys: see attn_bound)
                assert ((o[34 * s + i, h].double() - w @ v).abs() <= 2.0 ** -15 * (w @ v.abs())).all(), (s, i, h)


def test_two_groups_replayed():
    """Captured and replayed while sequences shrink, against eager calls."""
    need_gpu()
    b = Batch([(40, 700)] * 64, 32, 8, 128, "f16", seed=22)
    q = torch.randn((b.n_tokens, 8, 128), generator=torch.Generator().manual_seed(8)).to(b.dtype).cuda()
    cache, batch = b.device(R)
    og, oe = (torch.empty(q.shape, dtype=torch.float16, device="cuda") for _ in range(2))
    n = R.attn_workspace_bytes(cache, batch, 8)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.attn(q, cache, batch, og, 0.1, 0, 0, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        R.attn(q, cache, batch, og, 0.1, 0, 0, ws)
    for i in range(4):
        batch.kv_len.copy_((b.kv_len.cuda() - 150 * i).to(torch.int32))
        R.attn(q, cache, batch, oe, 0.1, 0, 0, ws)
        torch.cuda.synchronize()
        og.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, oe), i


# (lens, heads, kv_heads, dim, page): every kernel, unsplit and split
FAR = [
    ([(1, 300), (1, 1), (1, 40)], 4, 2, 64, 16),
    ([(4, 900), (2, 2)], 8, 1, 128, 32),
    ([(1, 5000)], 8, 1, 64, 64),
    ([(3, 200)], 5, 1, 80, 4),
    ([(60, 500), (33, 33)], 8, 2, 128, 16),
    ([(40, 400)], 4, 2, 64, 64),
    ([(30, 200)], 2, 1, 256, 32),
    ([(40, 6000)], 8, 1, 128, 32),
    ([(40, 300)] * 64, 8, 8, 128, 64),
]


@pytest.mark.parametrize("kind,log_q,log_k,log_unit,scale", [
    ("f16", 6, 5, 0, 0.5), ("f16", 11, 11, 0, 0.5), ("f16", 12, 12, 2, 0.25), ("f16", 15, 15, 8, 2.0 ** -9), ("f16", 15, 15, 8, 1.0),
    ("bf16", 11, 11, 0, 0.5), ("bf16", 20, 20, 18, 2.0 ** -20), ("bf16", 20, 20, 18, 1.0), ("bf16", 62, 62, 102, 8.0)])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_scores_far_from_zero(case, kind, log_q, log_k, log_unit, scale):
    """Scores that are all near 1.875 * 2^(log_q + log_k), of either sign, and
    differ by whole units: element 0 makes the offset, 15 elements of -2 .. 2
    times 2^(log_unit / 2) the differences, so that every partial sum is a
    whole number of units below 2^24 and the scores are exact in fp32. What is
    left is the weights' arithmetic: c to a half step, c (s - m) + BIAS
    rounded once (at most 150 + 15 in size where the weight counts), or, up to
    |c m| = 2^12, one of its two terms rounded there; exp2 and the sums as in
    attn_bound; and weights below fp16's smallest, 2^-35 of the largest."""
    need_gpu()
    lens, heads, kv, dim, page = FAR[case]
    say(f"attn far {lens[:3]} {kind} 2^{log_q + log_k} unit 2^{log_unit} scale {scale}")
    b = Batch(lens, page, kv, dim, kind, seed=500 + case)
    g = torch.Generator().manual_seed(case)
    uq, uk = 2.0 ** (log_unit // 2), 2.0 ** (log_unit - log_unit // 2)

    def small(shape, unit, lead):
        x = torch.zeros(shape)
        x[..., 1:min(16, dim)] = torch.randint(-2, 3, (*shape[:-1], min(16, dim) - 1), generator=g) * unit
        x[..., 0] = lead
        return x.to(b.dtype)

    for sign in (1.0, -1.0):
        b.k = torch.where(b.used[:, None, :, None], small(b.k.shape, uk, 1.25 * 2.0 ** log_k), float("nan")).to(b.dtype)
        q = small((b.n_tokens, heads, dim), uq, sign * 1.5 * 2.0 ** log_q)
        ref, mag, _ = attn_exact(b, q, scale)
        top = float(b.v.double().nan_to_num(0).abs().max())
        L = max(t for _, t in lens)
        for out in ("f32", "same"):
            o = run(b, q, scale, out=out).double()
            rel = 2 * ((1.5 * 150 + 15) * 2.0 ** -24 + 2.0 ** -12 + 8 * 2.0 ** -23 + L * 2.0 ** -24)
            half = torch.finfo(b.dtype).eps / 2
            tol = (rel + (half if out == "same" and b.max_q * (heads // kv) > 16 else 0)) * mag + L * 2.0 ** -35 * top
            if out == "same":
                tol = tol + half * (ref.abs() + tol) + 2.0 ** -25
            bad = ~((o - ref).abs() <= tol)
            assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first {o[bad][0]} for {ref[bad][0]} ({sign} {out})"


# Calls that the documentation allows and the lists above do not hold: heads
# of every multiple of 8 among prompts, many heads on one kv head, the largest
# pages, tables far wider than their sequences, windows as large as an int.
WIDE = [
    ([(70, 130), (3, 9)], 4, 2, 136, 16, 0, 0, 2),
    ([(40, 200)], 2, 2, 200, 8, 33, 5, 2),
    ([(65, 65)], 2, 1, 248, 64, 0, 0, 2),
    ([(60, 300)], 4, 1, 8, 32, 0, 0, 2),
    ([(33, 90)], 2, 1, 104, 1, 0, 0, 2),
    ([(1, 300), (2, 40)], 1024, 1, 16, 16, 0, 0, 2),
    ([(1, 5000), (50, 4100)], 4, 2, 64, 4096, 0, 0, 1),
    ([(3, 90), (1, 700)], 8, 2, 128, 16, 0, 0, 9000),
    ([(100, 100), (7, 400)], 8, 2, 128, 16, 0, 0, 9000),
    ([(100, 100)], 4, 2, 128, 1, 0, 0, 5000),
    ([(40, 40)] * 64, 8, 8, 128, 16, 0, 0, 4090),
    ([(40, 40)] * 64, 8, 8, 128, 16, 0, 0, 4100),
    ([(5, 300), (90, 200)], 4, 2, 64, 16, (1 << 31) - 1, (1 << 31) - 1, 2),
    ([(2, 300), (1, 200)], 4, 2, 64, 16, (1 << 31) - 1, 7, 2),
    ([(2, 300), (70, 200)], 4, 2, 64, 16, 5, (1 << 31) - 1, 2),
]


@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_wide_range(case, kind, out):
    lens, heads, kv, dim, page, window, sinks, more = WIDE[case]
    check(lens, heads, kv, dim, page, kind, window, sinks, out=out, seed=600 + case, extra_entries=more, tail=1)


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_query_that_is_not_finite(rows, value):
    """One query head with NaN or an infinity makes its own result NaN and
    leaves every other as it is."""
    need_gpu()
    b = Batch([(rows, 700), (rows, 90)], 16, 2, 64, "bf16", seed=15)
    q = torch.randn((2 * rows, 8, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    ref, mag, dots = attn_exact(b, q, 0.125)
    q[rows // 2, 3, 5] = value
    o = run(b, q, 0.125)
    assert torch.isnan(o[rows // 2, 3]).all()
    ok = (o.double() - ref).abs() <= attn_bound(b, ref, mag, dots, o.dtype, False)
    ok[rows // 2, 3] = True
    assert ok.all()


@pytest.mark.parametrize("rows", [1, 40])
def test_two_calls_at_once(rows):
    """Two calls on two streams, each with its workspace, over one cache."""
    need_gpu()
    b = Batch([(rows, 3000)], 32, 1, 64, "f16", seed=16)
    cache, batch = b.device(R)
    n = R.attn_workspace_bytes(cache, batch, 8)
    assert n > 0
    q = [torch.randn((rows, 8, 64), generator=torch.Generator().manual_seed(i)).to(b.dtype).cuda() for i in range(2)]
    want = [run(b, x, 0.125) for x in q]
    cache, batch = b.device(R)
    o = [torch.empty((rows, 8, 64), device="cuda") for _ in q]
    ws = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            R.attn(q[i], cache, batch, o[i], 0.125, 0, 0, ws[i], stream=s)
    torch.cuda.synchronize()
    for got, w in zip(o, want):
        assert torch.equal(got.cpu(), w)


def test_sequences_that_share_pages():
    """A common beginning: two sequences name the same pages, one a page
    twice."""
    need_gpu()
    b = Batch([(2, 100), (40, 140)], 16, 2, 64, "bf16", seed=17)
    b.table[0, :4] = b.table[1, :4]
    b.table[1, 6] = b.table[1, 2]
    q = torch.randn((42, 4, 64), generator=torch.Generator().manual_seed(8)).to(b.dtype)
    o = run(b, q, 0.125)
    ref, mag, dots = attn_exact(b, q, 0.125)
    assert ((o.double() - ref).abs() <= attn_bound(b, ref, mag, dots, o.dtype, False)).all()
