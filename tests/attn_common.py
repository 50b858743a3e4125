"""Helpers of the paged-attention tests: batches with their own pages in
random order, NaN in every slot that holds no token and ids out of range in
every table entry that no token needs, and the operators' definitions in 64
bits with elementwise error bounds."""

import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """lens: (new, total) tokens per sequence; `lead` rows of no sequence
    before the first and `tail` behind the last."""

    def __init__(self, lens, page, kv_heads, dim, kind, seed=0, lead=0, tail=0, extra_entries=2, max_q=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.kv_heads, self.dim, self.dtype = lens, page, kv_heads, dim, TYPES[kind]
        need = [-(-max(t, 0) // page) for _, t in lens]
        self.n_pages = max(1, sum(need)) + 2
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        stride = max(max(need), 1) + extra_entries
        bad = [-1, self.n_pages, 1 << 30, -(1 << 31)]
        table = [[bad[(s + j) % 4] for j in range(stride)] for s in range(len(lens))]
        at = 0
        for s, n in enumerate(need):
            table[s][:n] = ids[at:at + n]
            at += n
        self.table = torch.tensor(table, dtype=torch.int32)
        off = [lead]
        for n, _ in lens:
            off.append(off[-1] + n)
        self.q_off = torch.tensor(off, dtype=torch.int32)
        self.kv_len = torch.tensor([t for _, t in lens], dtype=torch.int32)
        self.n_tokens = off[-1] + tail
        self.max_q = max_q or max(1, max(n for n, _ in lens))
        shape = (self.n_pages, kv_heads, page, dim)
        self.k = torch.randn(shape, generator=g).to(self.dtype)
        self.v = torch.randn(shape, generator=g).to(self.dtype)
        used = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for s, (_, t) in enumerate(lens):
            for p in range(t):
                used[table[s][p // page], p % page] = True
        self.used = used
        for c in (self.k, self.v):
            c.masked_fill_(~used[:, None, :, None], float("nan"))

    def rows(self):
        """(row, sequence, position) of every new token."""
        return [(int(self.q_off[s]) + i, s, t - n + i) for s, (n, t) in enumerate(self.lens) for i in range(n)]

    def device(self, R):
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        self.cache = R.DeviceKVCache(self.kd, self.vd)
        self.batch = R.KVBatch(self.q_off.cuda(), self.kv_len.cuda(), self.table.cuda(), self.n_tokens, self.max_q)
        return self.cache, self.batch

    def keys(self, s, total):
        """[total][kv_heads][dim] of sequence s, in 64 bits."""
        page = torch.tensor([int(self.table[s, p // self.page]) for p in range(total)], dtype=torch.long)
        slot = torch.arange(total) % self.page
        return self.k[page, :, slot].double(), self.v[page, :, slot].double()


def attn_exact(b, q, scale, window=0, sinks=0):
    """(out, sum of p |v|, largest sum of |q_i k_i| scale) in 64 bits, out
    [n_tokens][heads][dim], NaN in rows of no sequence."""
    heads = q.shape[1]
    G = heads // b.kv_heads
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    mag = torch.zeros(q.shape, dtype=torch.float64)
    dots = 0.0
    for s, (n, total) in enumerate(b.lens):
        if n == 0:
            continue
        t0 = int(b.q_off[s])
        k, v = b.keys(s, max(total, 0))
        pos = torch.arange(total - n, total)[:, None]
        key = torch.arange(max(total, 0))[None]
        seen = key <= pos
        if window:
            seen = seen & ((key > pos - window) | (key < sinks))
        qs = q[t0:t0 + n].double()
        for h in range(heads):
            kk, vv = k[:, h // G], v[:, h // G]
            # keys and values that no row sees may hold anything
            any_row = seen.any(0)
            kk = torch.where(any_row[:, None], kk, 0.0)
            vv = torch.where(any_row[:, None], vv, 0.0)
            z = (qs[:, h] @ kk.t() * scale).masked_fill(~seen, -math.inf)
            dots = max(dots, float((qs[:, h].abs() @ kk.abs().t() * scale).max()) if kk.numel() else 0.0)
            top = z.amax(-1, keepdim=True) if z.shape[1] else torch.full((n, 1), -math.inf, dtype=torch.float64)
            p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            tot = p.sum(-1, keepdim=True)
            p = p / torch.where(tot == 0, 1.0, tot)
            out[t0:t0 + n, h] = p @ vv
            mag[t0:t0 + n, h] = p @ vv.abs()
    return out, mag, dots


def attn_bound(b, out, mag, dots, out_dtype, one_term):
    """Elementwise bound on the kernel's error. A weight p = exp2(c s - c m)
    is off, relatively, by the scores' error: each fp32 score is a sum of
    dim products in any order (dim half steps of 2^-24 of sum |q k|) and c s,
    c m are rounded once each (at most the same magnitude): ds = (dim + 8)
    2^-24 dots. exp2's own error and the rescaling of running sums are a few
    2^-23, the sums over L keys L half steps, all of sum p |v|, and again in
    the divisor. Weights carried as one 16-bit value add a half step. The
    result's own rounding is a half step of it (plus, for fp16, half the
    smallest subnormal)."""
    L = max([t for _, t in b.lens] + [1])
    rel = 2 * ((b.dim + 8) * 2.0 ** -24 * dots + 8 * 2.0 ** -23 + L * 2.0 ** -24)
    half = torch.finfo(b.dtype).eps / 2
    if one_term:
        rel += half
    tol = rel * mag
    if out_dtype != torch.float32:
        tol = tol + half * (out.abs() + tol) + 2.0 ** -25
    return tol + 2.0 ** -100


def rotate_exact(x, weight, eps, pos, inv_freq, interleaved):
    """Norm and rotation of [T][heads][dim] in 64 bits, and the magnitude
    that each element's fp32 error is relative to (its pair's length)."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    r = 2 * len(inv_freq)
    t = pos.double()[:, None] * inv_freq.double()
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
    y, mag = x.clone(), x.abs()
    i = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = a * c - b * s, b * c + a * s
    mag[..., i[0]] = mag[..., i[1]] = torch.hypot(a, b)
    return y, mag
