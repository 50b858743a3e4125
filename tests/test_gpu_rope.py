"""rfx_qk_norm_rope against its definition in 64 bits: norms, both pair
layouts, partial rotation, far positions, strided rows, ragged batches, and
the appended cache with everything else in it untouched."""

import pytest
import torch

import bit_block_quantized_amd as R
from attn_common import TYPES, Batch, rotate_exact
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


def close(got, ref, mag, dtype):
    """Half a step of the result (fp16: at least half its smallest
    subnormal) and the fp32 arithmetic: the norm's sum of up to 256 squares
    (at most 2^-17 in any order, half of it after the root), angle, sine and
    cosine to 2^-22 and four roundings: 2^-16 of the pair's length."""
    half = torch.finfo(dtype).eps / 2
    tol = half * ref.abs() + (1 + half) * 2.0 ** -16 * mag + 2.0 ** -25
    return (got.double() - ref).abs() <= tol


def check(lens, heads, kv_heads, dim, rot, page, kind, pairs, norm, fused=False, seed=0, base=10000.0, **kw):
    need_gpu()
    say(f"rope {lens[:4]} h={heads}/{kv_heads} d={dim} rot={rot} page={page} {kind} pairs={pairs} norm={norm}")
    b = Batch(lens, page, kv_heads, dim, kind, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    T = b.n_tokens
    qkv = torch.randn((T, heads + 2 * kv_heads, dim), generator=g) * 3
    wq = 1 + 0.2 * torch.randn(dim, generator=g) if norm else None
    wk = 1 + 0.2 * torch.randn(dim, generator=g) if norm else None
    inv = torch.from_numpy(R.rope_inv_freq(rot, base))
    before = b.k.clone(), b.v.clone()
    cache, batch = b.device(R)
    d = qkv.cuda()
    parts = d.split((heads, kv_heads, kv_heads), 1)
    if not fused:
        parts = [p.contiguous() for p in parts]
    out = torch.full((T, heads, dim), 7.0, dtype=b.dtype, device="cuda")
    R.qk_norm_rope(*parts, cache, batch, out, inv.cuda(), None if wq is None else wq.cuda(),
                   None if wk is None else wk.cuda(), 1e-5, pairs)
    torch.cuda.synchronize()
    out, k, v = out.cpu(), b.kd.cpu(), b.vd.cpu()
    rows = b.rows()
    idle = torch.ones(T, dtype=torch.bool)
    want_k, want_v = before
    put = torch.zeros((b.n_pages, page), dtype=torch.bool)
    if rows:
        at = torch.tensor([r for r, _, _ in rows])
        pos = torch.tensor([p for _, _, p in rows])
        idle[at] = False
        ref, mag = rotate_exact(qkv[at, :heads], wq, 1e-5, pos, inv, pairs)
        assert close(out[at], ref, mag, b.dtype).all()
        keep = pos >= 0
        at, pos = at[keep], pos[keep]
        ref, mag = rotate_exact(qkv[at, heads:heads + kv_heads], wk, 1e-5, pos, inv, pairs)
        ids = torch.tensor([int(b.table[s, p // page]) for _, s, p in rows if p >= 0], dtype=torch.long)
        assert close(k[ids, :, pos % page], ref, mag, b.dtype).all()
        assert torch.equal(v[ids, :, pos % page], qkv[at, heads + kv_heads:].to(b.dtype))
        put[ids, pos % page] = True
    assert (out[idle] == 7).all(), "rows of no sequence were written"
    rest = ~put[:, None, :, None].expand(k.shape)
    for got, want in ((k, want_k), (v, want_v)):
        assert torch.equal(got[rest].nan_to_num(99.0), want[rest].nan_to_num(99.0)), "other cache slots changed"


CASES = [
    ([(1, 1)], 1, 1, 8, 8, 1),
    ([(1, 100)], 32, 8, 128, 128, 16),
    ([(4, 4), (4, 700), (2, 65)], 16, 2, 64, 32, 64),
    ([(3, 50), (0, 20), (1, 0), (7, 5)], 6, 3, 80, 40, 8),
    ([(33, 33), (1, 900)], 5, 5, 256, 64, 32),
    ([(9, 30)], 8, 1, 200, 200, 4),
    ([(2, 77)], 3, 1, 120, 0, 2),
    ([(1, 40)] * 70, 4, 4, 64, 64, 16),
    ([(600, 650)], 2, 1, 64, 64, 256),
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_rotate_append(case, pairs, kind):
    lens, heads, kv, dim, rot, page = CASES[case]
    check(lens, heads, kv, dim, rot, page, kind, pairs, norm=case % 3 != 2, fused=case % 2 == 0, seed=case,
          lead=case % 2, tail=case % 3)


def test_many_sequences():
    """More sequences than one probe of 64 covers, some without new tokens."""
    check([(i % 3, 5 + i % 7) for i in range(5000)], 1, 1, 8, 8, 8, "bf16", False, True, lead=2, tail=3)


def test_far_positions():
    """Positions near 2^20 and a slow base: the angle is exact to 2^-30."""
    need_gpu()
    total = 1 << 20
    inv = torch.from_numpy(R.rope_inv_freq(64, 1e6))
    k = torch.zeros((total // 4096, 1, 4096, 64), dtype=torch.float16, device="cuda")
    cache = R.DeviceKVCache(k, torch.zeros_like(k))
    table = torch.arange(total // 4096, dtype=torch.int32, device="cuda")[None].contiguous()
    batch = R.KVBatch(torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                      torch.tensor([total], dtype=torch.int32, device="cuda"), table, 5, 5)
    x = torch.randn((5, 1, 64), generator=torch.Generator().manual_seed(1))
    out = torch.empty((5, 1, 64), dtype=torch.float16, device="cuda")
    R.qk_norm_rope(x.cuda(), x.cuda(), x.cuda(), cache, batch, out, inv.cuda())
    pos = torch.arange(total - 5, total)
    ref, mag = rotate_exact(x, None, 0.0, pos, inv, False)
    assert close(out.cpu(), ref, mag, torch.float16).all()
    assert close(k.reshape(total, 1, 64)[-5:].cpu(), ref, mag, torch.float16).all()


def test_bad_page_or_position_is_not_written():
    need_gpu()
    b = Batch([(2, 20), (2, 500)], 8, 1, 64, "bf16", seed=3)
    b.table[0, 2] = b.n_pages      # positions 18 and 19: no such page
    b.kv_len[1] = 8 * b.table.shape[1] + 2  # positions past the table
    cache, batch = b.device(R)
    x = torch.randn((4, 1, 64)).cuda()
    out = torch.empty((4, 1, 64), dtype=b.dtype, device="cuda")
    R.qk_norm_rope(x, x, x, cache, batch, out, torch.from_numpy(R.rope_inv_freq(64)).cuda())
    assert torch.equal(b.kd.cpu().nan_to_num(9.0), b.k.nan_to_num(9.0))
    assert torch.equal(b.vd.cpu().nan_to_num(9.0), b.v.nan_to_num(9.0))


def test_append_then_attend():
    """A decode loop as a program runs it: append, then attention over the
    grown cache, three steps of up to four tokens, against one prompt pass
    over all the tokens."""
    need_gpu()
    H, K, D, page, steps = 8, 2, 64, 16, (5, 4, 1, 3)
    T = sum(steps)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((T, H + 2 * K, D), generator=g).cuda()
    inv = torch.from_numpy(R.rope_inv_freq(D)).cuda()
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")

    def cache():
        return R.DeviceKVCache(*(torch.full((3, K, page, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)))

    def step(c, lo, n):
        batch = R.KVBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([lo + n], dtype=torch.int32, device="cuda"), table, n, n)
        q, o = torch.empty((n, H, D), dtype=torch.float16, device="cuda"), torch.empty((n, H, D), device="cuda")
        R.qk_norm_rope(*qkv[lo:lo + n].split((H, K, K), 1), c, batch, q, inv)
        ws = torch.zeros(max(1, R.attn_workspace_bytes(c, batch, H)), dtype=torch.uint8, device="cuda")
        R.attn(q, c, batch, o, 0.125, ws=ws)
        return o

    c, at, outs = cache(), 0, []
    for n in steps:
        outs.append(step(c, at, n))
        at += n
    full = step(cache(), 0, T)
    # both are within attn_bound of the definition (scores below 20, 13 keys): 2^-14 between them
    assert torch.allclose(torch.cat(outs), full, rtol=0, atol=2.0 ** -14 * 5)


@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("over", [1, 3, 1 << 30, (1 << 31) - 1 - 64])
def test_append_and_attention_agree_on_sequences(new, over):
    """Sequences whose tokens leave their table, or whose rows leave the
    arrays, are skipped by the append and by attention alike; the others, with
    negative positions among them, are served."""
    need_gpu()
    H, K, D, page, width = 4, 2, 64, 16, 4
    room = width * page
    lens = [(new, 50), (new, room), (new, new - 1), (new, 60), (new, 33)]
    b = Batch(lens, page, K, D, "bf16", seed=5, extra_entries=0)
    assert b.table.shape[1] == width
    b.table[:] = torch.arange(5 * width, dtype=torch.int32).view(5, width)  # every entry is a page
    b.n_pages = 5 * width
    b.k, b.v = (torch.randn((b.n_pages, K, page, D), generator=torch.Generator().manual_seed(7 + i)).to(b.dtype) for i in range(2))
    b.kv_len[1] = room + over
    b.n_tokens -= 1  # the last sequence's last row is outside
    cache, batch = b.device(R)
    T = b.n_tokens
    x = torch.randn((T, H + 2 * K, D), generator=torch.Generator().manual_seed(8))
    inv = torch.from_numpy(R.rope_inv_freq(D))
    q16 = torch.full((T, H, D), 7.0, dtype=b.dtype, device="cuda")
    R.qk_norm_rope(*x.cuda().split((H, K, K), 1), cache, batch, q16, inv.cuda())
    pos = torch.tensor([t - new + i for _, t in lens for i in range(new)])[:T]
    seq = torch.arange(5).repeat_interleave(new)[:T]
    live = (seq == 0) | (seq == 2) | (seq == 3)
    ref, mag = rotate_exact(x[:, :H], None, 0.0, pos, inv, False)
    out = q16.cpu()
    assert close(out[live], ref[live], mag[live], b.dtype).all() and (out[~live] == 7).all()
    put = live & (pos >= 0)
    want = b.k.clone(), b.v.clone()
    ref, mag = rotate_exact(x[:, H:H + K], None, 0.0, pos, inv, False)
    ids, slot = b.table[seq[put], pos[put] // page].long(), pos[put] % page
    k, v = b.kd.cpu(), b.vd.cpu()
    assert close(k[ids, :, slot], ref[put], mag[put], b.dtype).all()
    want[0][ids, :, slot] = k[ids, :, slot]
    want[1][ids, :, slot] = x[put, H + K:].to(b.dtype)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]), "other cache slots changed"
    o = torch.full((T, H, D), 7.0, device="cuda")
    n = R.attn_workspace_bytes(cache, batch, H)
    R.attn(q16, cache, batch, o, 0.125, ws=torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None)
    o = o.cpu()
    assert (o[~live] == 7).all() and not o[live & (pos < 0)].any()
    for s in (0, 2, 3):
        for i in (0, new - 1):
            r, p = s * new + i, lens[s][1] - new + i
            if p < 0:
                continue
            j = torch.arange(p + 1)
            page_of, at = b.table[s, j // page].long(), j % page
            for h in (0, H - 1):
                kk, vv = (c[page_of, h // 2, at].double() for c in (k, v))
                w = torch.softmax(kk @ out[r, h].double() * 0.125, 0)
                # attn_bound's terms: 2 (72 * 20 + 16 + 64) 2^-24 with sums of |q k| / 8 below 20, 64 products and keys
                assert ((o[r, h].double() - w @ vv).abs() <= 2.0 ** -12 * (w @ vv.abs())).all(), (s, i, h)
