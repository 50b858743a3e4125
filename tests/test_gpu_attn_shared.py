"""rfx_attn_shared against attention's definition in 64 bits: groups of every
size, prefixes that end inside pages and tiles, sequences of no group, and
groups that the arrays do not let share. To see that a prefix is read from the
first sequence's pages, the others' hold NaN in its places and their tables ids
out of range (which a caller's do not)."""

import math

import pytest
import torch

import bit_block_quantized_amd as R
from attn_common import TYPES, Batch, attn_bound, attn_exact
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


class SharedBatch(Batch):
    """groups: (prefix, [(new, total) of each sequence]); prefix None: the
    sequences are in no group (the first or the last groups only). copies: the
    other sequences' tables repeat the prefix's whole pages; whole: and their
    own pages have copies of its other tokens."""

    def __init__(self, groups, page, kv_heads, dim, kind, seed=0, copies=False, whole=False, **kw):
        lens = [s for _, seqs in groups for s in seqs]
        super().__init__(lens, page, kv_heads, dim, kind, seed=seed, **kw)
        self.first, self.prefix, self.off, self.len = {}, {}, [], []
        at = 0
        for p, seqs in groups:
            if p is not None:
                if not self.off:
                    self.off = [at]
                self.off.append(at + len(seqs))
                self.len.append(p)
                for s in range(at + 1, at + len(seqs)):
                    n, total = lens[s]
                    if p > 0 and total - n >= p: # shares: its own slots there are no tokens
                        self.first[s], self.prefix[s] = at, p
                        for j in range(p):
                            to, of, i = int(self.table[s, j // page]), int(self.table[at, j // page]), j % page
                            for c in (self.k, self.v):
                                c[to, :, i] = c[of, :, i] if whole else float("nan")
                        for j in range(p // page):
                            self.table[s, j] = self.table[at, j] if copies or whole else (-1, 1 << 30)[j % 2]
            at += len(seqs)
        self.most = max(int(self.q_off[b] - self.q_off[a]) for a, b in zip(self.off, self.off[1:]))

    def keys(self, s, total):
        if s not in self.first:
            return super().keys(s, total)
        p, slot = self.prefix[s], torch.arange(total) % self.page
        page = [int(self.table[self.first[s] if j < p else s, j // self.page]) for j in range(total)]
        page = torch.tensor(page, dtype=torch.long)
        return self.k[page, :, slot].double(), self.v[page, :, slot].double()

    def share(self, max_tokens=None, max_len=None):
        i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return R.KVPrefix(i(self.off), i(self.len), max_tokens or max(1, self.most), max_len or max(1, max(self.len)))


def run(b, q, scale, out="f32", **kw):
    cache, batch = b.device(R)
    pre = b.share(**kw)
    o = torch.full(q.shape, 7.0, dtype=torch.float32 if out == "f32" else b.dtype, device="cuda")
    n = R.attn_shared_workspace_bytes(cache, batch, pre, q.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None # NaN: it needs no initialisation
    R.attn_shared(q.cuda(), cache, batch, pre, o, scale, ws)
    torch.cuda.synchronize()
    return o.cpu()


def compare(b, q, o, scale, out, one_term):
    ref, mag, dots = attn_exact(b, q, scale)
    # joining two parts: a factor, a product and a sum more on either side
    tol = attn_bound(b, ref, mag, dots, o.dtype, one_term) + 8 * 2.0 ** -24 * mag
    idle = torch.isnan(ref)
    assert torch.equal(o.double()[idle], torch.full_like(ref, 7.0)[idle]), "rows of no sequence were written"
    bad = ~((o.double() - ref).abs() <= tol) & ~idle
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside: {(o.double() - ref).abs()[bad].max()} at {bad.nonzero()[0].tolist()}"


def check(groups, heads, kv_heads, dim, page, kind, out="f32", seed=0, scale=None, share=None, **kw):
    need_gpu()
    say(f"shared {[(p, len(s)) for p, s in groups]} h={heads}/{kv_heads} d={dim} page={page} {kind} -> {out}")
    b = SharedBatch(groups, page, kv_heads, dim, kind, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((b.n_tokens, heads, dim), generator=g).to(TYPES[kind])
    scale = dim ** -0.5 if scale is None else scale
    o = run(b, q, scale, out, **(share or {}))
    # one term a weight: a prefix of many rows, or rfx_attn's prompts
    G = heads // kv_heads
    rows = (share or {}).get("max_tokens", b.most) * G
    compare(b, q, o, scale, out, out != "f32" and (rows > 96 or b.max_q * G > 16))
    return b, q, o


# (groups, heads, kv_heads, dim, page): one sequence to many, prefixes from
# one token to thousands, ends inside pages and tiles, every head-dim class
CASES = [
    ([(1, [(1, 2), (1, 3)])], 4, 4, 64, 16),
    ([(32, [(1, 33), (1, 40), (1, 64)])], 8, 2, 128, 16),
    ([(100, [(1, 101)])], 8, 2, 128, 32),
    ([(500, [(1, 560), (1, 501), (1, 532), (1, 530)])], 32, 8, 128, 16),
    ([(37, [(4, 41), (2, 60), (0, 50), (3, 200)]), (130, [(4, 140), (1, 131)])], 8, 1, 128, 64),
    ([(333, [(2, 340), (1, 700), (4, 337)]), (0, [(1, 5)]), (64, [(1, 65)] * 3)], 5, 1, 80, 8),
    ([(70, [(1, 80), (1, 71), (2, 90)])], 8, 2, 256, 32),
    ([(1000, [(1, 1010)] * 7)], 16, 1, 256, 4),
    ([(77, [(1, 90)] * 20)], 20, 4, 120, 2),
    ([(301, [(1, 302 + 5 * i) for i in range(70)])], 4, 4, 64, 1),
    ([(257, [(4, 300 + i) for i in range(20)]), (64, [(4, 70)] * 3)], 8, 1, 128, 64),
    ([(2500, [(1, 2501 + 40 * i) for i in range(30)])], 16, 4, 128, 16),
    ([(190, [(2, 200 + i) for i in range(40)])], 4, 2, 200, 256),
    ([(6000, [(1, 6100), (1, 9000)])], 4, 1, 128, 128),
    ([(129, [(1, 200)] * 34)], 16, 2, 64, 16),
    ([(90, [(1, 100), (2, 93)] * 12)], 16, 4, 8, 32),
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_groups(case, kind):
    check(*CASES[case], kind, seed=case, lead=case % 2, tail=case % 3, copies=case % 2 == 0)
    check(*CASES[case], kind, out="same", seed=100 + case)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if c > 3])
def test_groups_as_if_their_prefixes_were_long(case, kind):
    """max_len says how long: their keys are split as a long prefix's."""
    for i, out in enumerate(("f32", "same")):
        check(*CASES[case], kind, out=out, seed=200 + case, lead=i, share=dict(max_len=1 << 20))


@pytest.mark.parametrize("heads,kv_heads", [(4, 1), (32, 2)])
def test_sequences_of_no_group(heads, kv_heads):
    """Before the first group and behind the last, with and without splits."""
    groups = [(None, [(1, 40), (2, 1500)]), (200, [(1, 201), (2, 260)]), (None, [(1, 1), (0, 9), (1, 700)])]
    check(groups, heads, kv_heads, 128, 16, "bf16", lead=2, tail=1)
    check([(None, [(1, 2000)])] + [(50, [(1, 60), (1, 51)])], 4, 1, 64, 64, "f16", out="same")


def test_what_cannot_be_shared_is_attended_alone():
    """New tokens that begin inside the prefix, groups of more tokens than
    max_tokens, prefixes that are not positive or leave the table, sequences
    that leave the batch: each over its own pages."""
    check([(100, [(2, 150), (4, 102), (1, 100), (1, 101), (3, 50)])], 8, 2, 128, 16, "bf16", whole=True)
    for p in (0, -5, 1 << 30, 2 ** 31 - 1, -2 ** 31):
        check([(p, [(1, 40), (2, 77)])], 8, 2, 128, 16, "bf16", share=dict(max_len=100))
    need_gpu()
    b = Batch([(2, 90), (1, 150), (1, 33)], 16, 2, 64, "f16", seed=5)
    q = torch.randn((4, 8, 64), generator=torch.Generator().manual_seed(6)).half()
    ref, mag, dots = attn_exact(b, q, 0.125)
    tol = attn_bound(b, ref, mag, dots, torch.float32, False)
    cache, batch = b.device(R)
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for off, length, most in (([0, 3], [32], 3), ([0, 4], [32], 9), ([-1, 3], [32], 9), ([2, 1], [16], 9), ([3, 5], [16], 9),
                              ([-2 ** 31, 2 ** 31 - 1], [16], 9), ([0, 0, 0], [5, 5], 9), ([5, -5, 5, 1], [9, 9, 9], 9)):
        say(f"seq_off {off}")
        pre = R.KVPrefix(i(off), i(length), most, 64)
        o = torch.empty((4, 8, 64), device="cuda")
        n = R.attn_shared_workspace_bytes(cache, batch, pre, 8)
        R.attn_shared(q.cuda(), cache, batch, pre, o, 0.125, torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
        assert ((o.cpu().double() - ref).abs() <= tol).all(), off


def test_more_rows_than_the_decode_kernel_takes():
    for kind in ("bf16", "f16"):
        b, _, _ = check([(100, [(40, 150), (3, 103)]), (64, [(20, 200)])], 4, 2, 128, 16, kind, whole=True)
        assert b.max_q * 2 > 32


def test_bad_pages_of_a_prefix_are_not_seen():
    """An unusable page of the first sequence's table hides its keys from the
    whole group, as rfx_attn hides them from the sequence."""
    need_gpu()
    for heads, n in ((8, 3), (8, 40)):
        b = SharedBatch([(96, [(1, 100 + i) for i in range(n)])], 16, 2, 64, "bf16", seed=3)
        q = torch.randn((b.n_tokens, heads, 64), generator=torch.Generator().manual_seed(4)).bfloat16()
        good = int(b.table[0, 2])
        b.table[0, 2] = b.n_pages + 7
        o = run(b, q, 0.125)
        # the definition over the keys that are left
        b.table[0, 2] = good
        keep = [j for j in range(200) if not 32 <= j < 48]
        for s, (_, total) in enumerate(b.lens):
            k, v = b.keys(s, total)
            on = [j for j in keep if j < total]
            for h in range(heads):
                z = q[s, h].double() @ k[on, h // (heads // 2)].t() * 0.125
                want = torch.softmax(z, -1) @ v[on, h // (heads // 2)]
                assert ((o[s, h].double() - want).abs() <= 2e-5 * v[on].abs().max()).all(), (s, h)


def test_scores_far_from_zero():
    for kind in ("f16", "bf16"):
        for scale in (40.0, 1e-6):
            check([(200, [(1, 230), (1, 260), (2, 202)]), (300, [(1, 301 + i) for i in range(40)])], 8, 2, 64, 32, kind, scale=scale)


def test_wrong_hints_do_not_matter():
    """max_len and max_tokens beyond what the arrays hold."""
    groups = [(700, [(1, 720 + i) for i in range(10)])]
    for share in (dict(max_len=1), dict(max_len=1 << 20), dict(max_tokens=400), dict(max_tokens=3)):
        # ten new tokens, past a max_tokens of three: one by one
        check(groups, 8, 2, 128, 32, "bf16", share=share, whole=share.get("max_tokens") == 3)


@pytest.mark.parametrize("n", [4, 40])
def test_captured_with_growing_sequences(n):
    torch = need_gpu()
    b = SharedBatch([(260, [(1, 300 + 3 * i) for i in range(n)])], 16, 2, 128, "bf16", seed=7)
    q = torch.randn((n, 16, 128), generator=torch.Generator().manual_seed(8)).bfloat16()
    cache, batch = b.device(R)
    pre, qd = b.share(), q.cuda()
    o = torch.empty((n, 16, 128), device="cuda")
    ws = torch.empty(R.attn_shared_workspace_bytes(cache, batch, pre, 16), dtype=torch.uint8, device="cuda")
    R.attn_shared(qd, cache, batch, pre, o, 0.09, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.attn_shared(qd, cache, batch, pre, o, 0.09, ws)
    for step in range(3):
        # shorter sequences, and a prefix of 256 or 260 tokens: the four between
        # are then read from each sequence's own pages
        p = (260, 256, 260)[step]
        b.lens = [(1, 262 + (7 * s + 11 * step) % 38) for s in range(n)]
        batch.kv_len.copy_(torch.tensor([t for _, t in b.lens]))
        pre.length.fill_(p)
        if p == 256:
            for s in b.prefix:
                b.prefix[s] = p
                own, first = int(b.table[s, 16]), int(b.table[0, 16])
                for c, d in ((b.k, b.kd), (b.v, b.vd)):
                    c[own, :, :4] = c[first, :, :4]
                    d.copy_(c)
        g.replay()
        torch.cuda.synchronize()
        compare(b, q, o.cpu(), 0.09, "f32", False)
        again = torch.empty_like(o)
        R.attn_shared(qd, cache, batch, pre, again, 0.09, ws)
        assert torch.equal(again, o)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [4, 40])
def test_weights_of_a_16_bit_result_are_whole(n, dim, kind):
    """Half of a prefix's keys have the weight 1 and the value 1, half have
    0.501953125 (or 0.500244140625), between two 16-bit values, and the value
    -2: nothing averages out what a weight is off by. Rounded to one value each
    the weights are off by 2^-8 (2^-11) of that, 2.6e-3 (3.3e-4) of a result
    whose bound here is below 1e-4. Four sequences' rows and forty's, which
    take another kernel, are held to the same bound."""
    need_gpu()
    say(f"whole weights {n} sequences, heads of {dim}, {kind}")
    b = SharedBatch([(200, [(1, 203)] * n)], 16, 2, dim, kind, seed=n)
    w = 0.5 * (1 + (2.0 ** -8 if kind == "bf16" else 2.0 ** -11))
    for t in (b.k, b.v):
        t.copy_(torch.where(torch.isnan(t), t, torch.zeros_like(t)))
    b.k[..., 0] = torch.where(torch.isnan(b.k[..., 0]), b.k[..., 0], torch.full_like(b.k[..., 0], -1.0))
    for j in range(200):
        page, slot = int(b.table[0, j // 16]), j % 16
        b.k[page, :, slot, 0] = 0.0 if j % 2 else -1.0
        b.v[page, :, slot] = 1.0 if j % 2 else -2.0
    q = torch.zeros((n, 8, dim), dtype=TYPES[kind])
    q[..., 0] = 1
    scale = -math.log(w)
    compare(b, q, run(b, q, scale, "same"), scale, "same", False)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("first", [(1, 40), (0, 40), (0, 0), (1, 99), (4, 99), (0, 5000)])
def test_a_first_sequence_without_the_prefix(first, n):
    """Its pages cannot be read for the group: whoever is in it is attended
    alone. The table behind its tokens names pages that others hold."""
    need_gpu()
    say(f"first sequence {first} of {n}")
    b = Batch([(first[0], min(first[1], 40 if first[1] > 100 else first[1]))] + [(1, 130 + i) for i in range(n)], 16, 2, 64, "bf16",
              seed=n)
    held = -(-int(b.kv_len[0]) // 16)
    b.table[0, held:] = b.table[1, :b.table.shape[1] - held].clamp(0, b.n_pages - 1)
    cache, batch = b.device(R)
    batch.kv_len[0] = first[1] # 5000 tokens leave the table
    q = torch.randn((b.n_tokens, 8, 64), generator=torch.Generator().manual_seed(n)).bfloat16()
    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pre = R.KVPrefix(i([0, n + 1]), i([100]), b.n_tokens, 100)
    o = torch.full(q.shape, 7.0, device="cuda")
    ws = torch.full((R.attn_shared_workspace_bytes(cache, batch, pre, 8),), 255, dtype=torch.uint8, device="cuda")
    R.attn_shared(q.cuda(), cache, batch, pre, o, 0.125, ws)
    compare(b, q, o.cpu(), 0.125, "f32", False)
    # a prefix that it has, to the last token or without a new one, is read from it
    for seqs in ([(1, 100)] + [(1, 101 + i) for i in range(n)], [(0, 99)] + [(1, 100 + i) for i in range(n)]):
        check([(99, seqs)], 8, 2, 64, 16, "bf16", copies=True)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("groups", [64, 65, 90, 300])
def test_many_groups(groups, kind):
    """More than a wave has lanes; some have no sequence, some no prefix."""
    seqs = lambda g: [(1 + (g + i) % 2, 60 + (7 * g + i) % 30) for i in range(g % 4)]  # noqa: E731
    many = [(-1 if g % 11 == 5 else 16 + g % 40, seqs(g)) for g in range(groups)]
    check([(None, [(1, 30)])] + many + [(None, [(2, 45), (1, 7)])], 8, 2, 64, 16, kind, seed=groups)
    check(many, 4, 1, 128, 32, kind, out="same", seed=groups + 1, share=dict(max_tokens=100))
