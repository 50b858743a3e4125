"""Measured cases of the attention half of a decoder layer and of the dense
projections around it: per-head norms of queries and keys with the position
rotation and the cache append ("rope"), attention over a paged key-value
cache for one to four new tokens per sequence and for prompts ("attn"), and
the product of packed block-quantized weights with bias, activation and
residual ("gemm").

run() computes the plain form (elementary torch operations in 32 bits) or,
with `own` set, calls the library.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
FMT = {"FP2": 2, "FP3": 3, "FP4": 4}
BLOCK_BYTES = {"FP2": 10, "FP3": 14, "FP4": 17}
TILE_BYTES = {"FP2": 5120, "FP3": 7168, "FP4": 8704}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of one sequence through the projections' outputs: the
        # smallest call of a decode step, where the launch itself counts
        dict(name="rope 1 token", op="rope", type="bf16", n_seq=1, q_max=1, ctx=1000, ragged=False, heads=32,
             kv_heads=8, dim=128, rot=128, pairs=False, norm=True, page=16),
        # four verification positions of each of 16 sequences, a quarter of
        # each head rotated, adjacent pairs
        dict(name="rope verify 16x4", op="rope", type="f16", n_seq=16, q_max=4, ctx=4000, ragged=False, heads=64,
             kv_heads=8, dim=64, rot=32, pairs=True, norm=False, page=64),
        # prompts of different lengths in one batch
        dict(name="rope prompts", op="rope", type="bf16", n_seq=5, q_max=4096, ctx=300, ragged=True, heads=32,
             kv_heads=8, dim=128, rot=128, pairs=False, norm=True, page=16),
        # one new token, one sequence: batch-one decode
        dict(name="decode 1x1", op="attn", type="bf16", out="f32", n_seq=1, q_max=1, ctx=1537, ragged=False, heads=32,
             kv_heads=8, dim=128, page=16, window=0, sinks=0),
        # four verification positions of eight sequences, contexts to 8192
        dict(name="decode verify 8x4", op="attn", type="f16", out="f32", n_seq=8, q_max=4, ctx=8188, ragged=True,
             heads=32, kv_heads=4, dim=128, page=64, window=0, sinks=0),
        # a serving batch over long contexts: the cache's bytes bound it
        dict(name="decode 32x1 long", op="attn", type="bf16", out="f32", n_seq=32, q_max=1, ctx=16384, ragged=True,
             heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a short chunk late in a long sequence, sliding window with sinks
        dict(name="chunk 100 window", op="attn", type="bf16", out="same", n_seq=1, q_max=100, ctx=5000, ragged=False,
             heads=32, kv_heads=8, dim=128, page=16, window=1024, sinks=4),
        # one long prompt, causal
        dict(name="prompt 8192", op="attn", type="bf16", out="same", n_seq=1, q_max=8192, ctx=0, ragged=False,
             heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # prompts of different lengths, sliding window with sinks, fp32 out
        dict(name="prompts window", op="attn", type="f16", out="f32", n_seq=6, q_max=4096, ctx=200, ragged=True,
             heads=32, kv_heads=8, dim=64, page=32, window=1024, sinks=4),
        # one column against a small FP4 matrix with bias and residual
        dict(name="gemm q1", op="gemm", fmt="FP4", q=1, rows=2048, cols=4096, bias=True, act="none", resid=True),
        # four verification columns, the dense benchmark's matrix
        dict(name="gemm q4", op="gemm", fmt="FP3", q=4, rows=7168, cols=7168, bias=False, act="silu", resid=True),
        # a prompt's projection
        dict(name="gemm q2048", op="gemm", fmt="FP4", q=2048, rows=4096, cols=7168, bias=True, act="gelu_tanh",
             resid=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rope", "decode", "prompt", "gemm", "gemv"))
    if op in ("gemm", "gemv"):
        return dict(op="gemm", fmt=rng.choice(("FP2", "FP3", "FP4")), q=rng.randint(1, 4) if op == "gemv" else _log(rng, 5, 2048),
                    rows=_log(rng, 33, 4096), cols=32 * _log(rng, 4, 224), bias=rng.random() < 0.5,
                    act=rng.choice(ACTS), resid=rng.random() < 0.5)
    heads = dict(kv_heads=rng.choice((1, 2, 4, 8)), dim=rng.choice((64, 80, 128, 128, 256)))
    heads["heads"] = heads["kv_heads"] * rng.choice((1, 2, 4, 8))
    kind = rng.choice(("bf16", "f16"))
    page = rng.choice((1, 8, 16, 32, 64, 256))
    ragged = rng.random() < 0.7
    if op == "rope":
        n_seq = _log(rng, 1, 40)
        return dict(op="rope", type=kind, n_seq=n_seq, q_max=_log(rng, 1, max(1, 8192 // n_seq)), ctx=_log(rng, 1, 3000),
                    ragged=ragged, rot=rng.choice((heads["dim"], heads["dim"] // 2 // 8 * 8)), pairs=rng.random() < 0.5,
                    norm=rng.random() < 0.7, page=page, **heads)
    window = rng.choice((0, 0, _log(rng, 1, 2000)))
    mask = dict(window=window, sinks=rng.choice((0, 1, 4, 31)) if window else 0)
    if op == "decode":
        n_seq = _log(rng, 1, 48)
        return dict(op="attn", type=kind, out=rng.choice(("f32", "same")), n_seq=n_seq, q_max=rng.randint(1, 4),
                    ctx=_log(rng, 1, 180000 // n_seq), ragged=ragged, page=page, **mask, **heads)
    n_seq = _log(rng, 1, 8)
    return dict(op="attn", type=kind, out=rng.choice(("f32", "same", "same")), n_seq=n_seq,
                q_max=_log(rng, 5, 2048 // n_seq), ctx=_log(rng, 1, 3000), ragged=ragged, page=page, **mask, **heads)


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the
    first at the case's bounds, the others, where the case is ragged, anywhere
    below, one of four or more with no new token."""
    rng = random.Random("%d %d %d" % (case["n_seq"], case["q_max"], case["ctx"]))
    new, total = [], []
    for s in range(case["n_seq"]):
        n, c = case["q_max"], case["ctx"]
        if case["ragged"] and s:
            n = 0 if s == 3 else rng.randint(max(1, n // 4), n)
            c = rng.randint(c // 2, c)
        new.append(n)
        total.append(c + n)
    return new, total


# ----------------------------------------------------------------- inputs

def _normal(gen, shape, sigma=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(sigma).to(dtype)


def _ints(gen, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=gen, device=DEV, dtype=dtype)


def _batch(case, gen):
    """The paged cache, a table of its pages in random order, and the
    sequences' offsets and lengths."""
    new, total = _lengths(case)
    page = case["page"]
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(new), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    shape = (n_pages, case["kv_heads"], page, case["dim"])
    t = TYPES[case["type"]]
    return dict(k_cache=_normal(gen, shape, dtype=t), v_cache=_normal(gen, shape, dtype=t), table=table,
                q_off=torch.tensor(off, dtype=torch.int32, device=DEV),
                kv_len=torch.tensor(total, dtype=torch.int32, device=DEV), tokens=off[-1])


def _weight(case, gen):
    """A packed matrix in the library's tiled layout with random codes and
    block scales about those of N(0, 0.02) weights; padding is zero."""
    fmt, rows, cols = case["fmt"], case["rows"], case["cols"]
    G, S = -(-rows // 64), -(-cols // 256)
    w = _ints(gen, 0, 256, (G, S, TILE_BYTES[fmt]), torch.uint8)
    if fmt == "FP4":
        w[:, :, 8192:] = _ints(gen, 117, 121, (G, S, 512), torch.uint8)
    else:
        n = 1024 * (4 if fmt == "FP2" else 6)
        amax = torch.rand((G, S, 512), generator=gen, device=DEV) * 0.04 + 0.02
        w[:, :, n:n + 1024] = (amax / (3 if fmt == "FP2" else 7)).to(torch.float16).view(torch.uint8)
    row_ok = (torch.arange(64 * G, device=DEV) < rows).reshape(G, 1, 64)
    blk_ok = (torch.arange(8 * S, device=DEV) < cols // 32).reshape(1, S, 8)
    ok = row_ok[..., None] & blk_ok[:, :, None, :]  # [G][S][64 rows][8 blocks]

    def clear(first, chunks, blocks_per_chunk, width):
        v = w[:, :, first:first + chunks * 1024].view(G, S, chunks, 64, blocks_per_chunk, width)
        m = ok.reshape(G, S, 64, chunks, blocks_per_chunk).permute(0, 1, 3, 2, 4)
        v.mul_(m[..., None].to(torch.uint8))

    if fmt == "FP4":
        clear(0, 8, 1, 16)
        w[:, :, 8192:].view(G, S, 64, 8).mul_(ok.to(torch.uint8))
    else:
        clear(0, 4, 2, 8)
        if fmt == "FP3":
            clear(4096, 2, 4, 4)
        clear(4096 if fmt == "FP2" else 6144, 1, 8, 2)
    return w.reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)
    st = dict(case=dict(case))
    if case["op"] == "gemm":
        q, N, K = case["q"], case["rows"], case["cols"]
        st["w"] = _weight(case, gen)
        # activations as a program holds them: int8 codes, a scale per 32, the codes' sums
        x = _normal(gen, (q, K // 32, 32))
        xs = x.abs().amax(-1) / 127
        xq = torch.round(x / xs[..., None]).clamp_(-127, 127)
        st["xq"] = xq.to(torch.int8).reshape(q, K)
        st["xs"] = xs.contiguous()
        st["xsum"] = xq.sum(-1).to(torch.int32)
        st["bias"] = _normal(gen, (N,), 0.5) if case["bias"] else None
        st["resid"] = _normal(gen, (q, N)) if case["resid"] else None
        st["y"] = torch.empty((q, N), dtype=torch.float32, device=DEV)
        if own:
            import bit_block_quantized_amd as R
            st["R"] = R
            st["W"] = R.DeviceQMat(FMT[case["fmt"]], N, K, st["w"])
            n = R.gemm_workspace_bytes(st["W"], q)
            st["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV) if n else None
            st["act"] = R.ACTIVATIONS[case["act"]]
        return st
    st.update(_batch(case, gen))
    T, Hq, Hk, D = st["tokens"], case["heads"], case["kv_heads"], case["dim"]
    t = TYPES[case["type"]]
    if case["op"] == "rope":
        # one fused projection's output: queries, keys and values side by side
        qkv = _normal(gen, (T, (Hq + 2 * Hk) * D))
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split((Hq * D, Hk * D, Hk * D), 1))
        st["wq"] = _normal(gen, (D,), 0.1).add_(1) if case["norm"] else None
        st["wk"] = _normal(gen, (D,), 0.1).add_(1) if case["norm"] else None
        half = case["rot"] // 2
        st["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        st["out"] = torch.empty((T, Hq, D), dtype=t, device=DEV)
    else:
        st["q"] = _normal(gen, (T, Hq, D), dtype=t)
        st["scale"] = 1 / math.sqrt(D)
        st["out"] = torch.empty((T, Hq, D), dtype=torch.float32 if case["out"] == "f32" else t, device=DEV)
    if own:
        import bit_block_quantized_amd as R
        st["R"] = R
        st["cache"] = R.DeviceKVCache(st["k_cache"], st["v_cache"])
        st["batch"] = R.KVBatch(st["q_off"], st["kv_len"], st["table"], T, case["q_max"])
        if case["op"] == "attn":
            n = R.attn_workspace_bytes(st["cache"], st["batch"], Hq)
            st["ws"] = torch.zeros(n, dtype=torch.uint8, device=DEV) if n else None
    return st


# ------------------------------------------------------------- plain forms

def _rows(st):
    """Sequence and position of each new token."""
    t = torch.arange(st["tokens"], device=DEV)
    s = torch.searchsorted(st["q_off"][1:].contiguous(), t.to(torch.int32), right=True)
    return s, t - st["q_off"][s + 1] + st["kv_len"][s]


def _norm_rotate(x, weight, cos, sin, rot, pairs):
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(st):
    case = st["case"]
    s, pos = _rows(st)
    angle = pos.double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    t, page = TYPES[case["type"]], case["page"]
    st["out"].copy_(_norm_rotate(st["q"], st["wq"], cos, sin, case["rot"], case["pairs"]))
    k = _norm_rotate(st["k"], st["wk"], cos, sin, case["rot"], case["pairs"])
    where = st["table"][s, pos // page].long()
    st["k_cache"][where, :, pos % page] = k.to(t)
    st["v_cache"][where, :, pos % page] = st["v"].to(t)
    return dict(q=st["out"], k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_attn(st):
    case = st["case"]
    n, mq, page = case["n_seq"], case["q_max"], case["page"]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G, L = Hq // Hk, st["table"].shape[1] * page
    # the sequences' caches and queries, padded to the longest
    ids = st["table"].long()
    k = st["k_cache"][ids].transpose(1, 2).reshape(n, Hk, L, D).float()
    v = st["v_cache"][ids].transpose(1, 2).reshape(n, Hk, L, D).float()
    new = st["q_off"][1:] - st["q_off"][:-1]
    i = torch.arange(mq, device=DEV)
    row = (st["q_off"][:-1, None] + i).clamp_(max=st["tokens"] - 1).long()
    q = st["q"][row].float().reshape(n, mq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hk, mq * G, D)
    pos = (st["kv_len"] - new)[:, None] + i
    j = torch.arange(L, device=DEV)
    seen = j <= pos[..., None]
    if case["window"]:
        seen &= (j > pos[..., None] - case["window"]) | (j < case["sinks"])
    score = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(n, Hk, mq, G, L)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, Hk, mq * G, L) @ v).view(n, Hk, mq, G, D) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(n * mq, Hq, D)
    s, at = _rows(st)
    st["out"].copy_(o[s * mq + at - pos[s, 0]])
    return st["out"]


def _plain_weights(case, w):
    fmt, rows, cols = case["fmt"], case["rows"], case["cols"]
    G, S = -(-rows // 64), -(-cols // 256)
    w = w.view(G, S, -1)
    if fmt == "FP4":
        b = w[:, :, :8192].view(G, S, 8, 64, 4, 4)  # [block][row][word m][byte j]
        code = torch.stack((b & 15, b >> 4), -2).reshape(G, S, 8, 64, 32)  # weight 8m + 4i + j
        value = torch.tensor([0., 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], device=DEV)[code.int()]
        e = w[:, :, 8192:].view(G, S, 64, 8).permute(0, 1, 3, 2)
        scale = torch.exp2(e.float() - 128)
    else:
        b = w[:, :, :4096].view(G, S, 4, 64, 2, 2, 4).permute(0, 1, 2, 4, 3, 5, 6).reshape(G, S, 8, 64, 2, 4)
        code = torch.stack([(b >> (2 * i)) & 3 for i in range(4)], -2).reshape(G, S, 8, 64, 32)  # 16m + 4i + j
        if fmt == "FP3":
            h = w[:, :, 4096:6144].view(G, S, 2, 64, 4, 4).permute(0, 1, 2, 4, 3, 5).reshape(G, S, 8, 64, 4)
            code = code | (torch.stack([(h >> i) & 1 for i in range(8)], -2) << 2).reshape(G, S, 8, 64, 32)
        value = 2 * code.float() - (3 if fmt == "FP2" else 7)
        n = 4096 if fmt == "FP2" else 6144
        scale = w[:, :, n:n + 1024].view(torch.float16).view(G, S, 64, 8).permute(0, 1, 3, 2).float()
    full = (value * scale[..., None]).permute(0, 3, 1, 2, 4).reshape(64 * G, 256 * S)
    return full[:rows, :cols]


def _plain_gemm(st):
    case = st["case"]
    q, K = case["q"], case["cols"]
    x = (st["xq"].float().view(q, K // 32, 32) * st["xs"][..., None]).view(q, K)
    y = x @ _plain_weights(case, st["w"]).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    act = case["act"]
    if act == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if st["resid"] is not None:
        y = y + st["resid"]
    return y


def run(st):
    op = st["case"]["op"]
    if not own:
        return (_plain_rope if op == "rope" else _plain_attn if op == "attn" else _plain_gemm)(st)
    R, case = st["R"], st["case"]
    if op == "rope":
        R.qk_norm_rope(st["q"], st["k"], st["v"], st["cache"], st["batch"], st["out"], st["inv_freq"], st["wq"],
                       st["wk"], EPS, case["pairs"])
        return dict(q=st["out"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    if op == "attn":
        R.attn(st["q"], st["cache"], st["batch"], st["out"], st["scale"], case["window"], case["sinks"], st["ws"])
        return st["out"]
    R.gemm(st["W"], st["xq"], st["xs"], st["xsum"], case["q"], st["y"], st["bias"], st["act"], st["resid"], st["ws"])
    return st["y"]


# -------------------------------------------------------------------- work

def _visible(case, p):
    """Keys that the token at position p sees."""
    if not case["window"]:
        return p + 1
    return min(p + 1, case["window"]) + min(case["sinks"], max(0, p + 1 - case["window"]))


def work(case):
    if case["op"] == "gemm":
        q, N, K = case["q"], case["rows"], case["cols"]
        return dict(bytes=N * K // 32 * BLOCK_BYTES[case["fmt"]] + q * (K + K // 4) + 4 * N * (q * (1 + case["resid"]) + case["bias"]),
                    flops=2 * q * N * K)
    new, total = _lengths(case)
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    T = sum(new)
    if case["op"] == "rope":
        n = T * (Hq + 2 * Hk) * D
        return dict(bytes=6 * n, flops=8 * n)
    keys = pairs = 0
    for n, c in zip(new, total):
        if n:
            first, w, sk = c - n, case["window"], case["sinks"]
            low = max(0, first - w + 1) if w else 0
            keys += c - low + min(sk, low)
            pairs += sum(_visible(case, p) for p in range(first, c))
    wide = 4 if case["out"] == "f32" else 2
    return dict(bytes=4 * keys * Hk * D + T * Hq * D * (2 + wide), flops=4 * pairs * Hq * D)


# ------------------------------------------------------- 64-bit definitions

def _exact_rope(case, st):
    t = st["tokens"]
    new, total = _lengths(case)
    pos = torch.tensor([p for n, c in zip(new, total) for p in range(c - n, c)], dtype=torch.float64, device=DEV)
    where = [(s, p) for s, (n, c) in enumerate(zip(new, total)) for p in range(c - n, c)]
    rot = case["rot"]
    turn = torch.polar(torch.ones((t, rot // 2), dtype=torch.float64, device=DEV), torch.outer(pos, st["inv_freq"]))

    def one(x, w):
        x = x.double()
        if w is not None:
            x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        y = x.clone()
        first = slice(0, rot, 2) if case["pairs"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["pairs"] else slice(rot // 2, rot)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    k, v = one(st["k"], st["wk"]), st["v"].double()
    table = st["table"].tolist()
    page = case["page"]
    ids = torch.tensor([table[s][p // page] for s, p in where], device=DEV)
    slot = torch.tensor([p % page for _, p in where], device=DEV)
    for h in range(case["kv_heads"]):
        kc[ids, h, slot], vc[ids, h, slot] = k[:, h], v[:, h]
    return dict(q=one(st["q"], st["wq"]), k_cache=kc, v_cache=vc)


def _exact_attn(case, st):
    new, total = _lengths(case)
    Hq, Hk, page = case["heads"], case["kv_heads"], case["page"]
    G = Hq // Hk
    out = torch.zeros((st["tokens"], Hq, case["dim"]), dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, c) in enumerate(zip(new, total)):
        ids = st["table"][s, :-(-c // page)].long()
        key = torch.arange(c, device=DEV)[None]
        for lo in range(0, n, 2048):  # a stretch of the new tokens at a time
            m = min(2048, n - lo)
            p = torch.arange(c - n + lo, c - n + lo + m, device=DEV)[:, None]
            hidden = key > p
            if case["window"]:
                hidden |= (key <= p - case["window"]) & (key >= case["sinks"])
            for h in range(Hk):
                k = st["k_cache"][ids, h].double().flatten(0, 1)[:c]
                v = st["v_cache"][ids, h].double().flatten(0, 1)[:c]
                for g in range(h * G, h * G + G):
                    z = torch.softmax((st["q"][at + lo:at + lo + m, g].double() @ k.t() * st["scale"]).masked_fill(hidden, -math.inf), -1)
                    out[at + lo:at + lo + m, g] = z @ v
        at += n
    return out


def _exact_weights(case, w):
    """Weight (r, c) from its own bits: byte and shift of every column of a
    256-column tile, then one gather."""
    fmt, rows, cols = case["fmt"], case["rows"], case["cols"]
    c = torch.arange(cols, device=DEV)
    r = torch.arange(rows, device=DEV)[:, None]
    tile = (r // 64) * -(-cols // 256) + c // 256
    b, t, lane = c % 256 // 32, c % 32, r % 64
    base = tile * TILE_BYTES[fmt]
    if fmt == "FP4":
        x = w[base + b * 1024 + lane * 16 + t // 8 * 4 + t % 4].int() >> (t // 4 % 2 * 4) & 15
        mag = torch.tensor([0., .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        value = torch.where(x < 8, mag[x % 8], -mag[x % 8])
        return value * torch.pow(2.0, w[base + 8192 + lane * 8 + b].double() - 127)
    x = w[base + b // 2 * 1024 + lane * 16 + b % 2 * 8 + t // 16 * 4 + t % 4].int() >> (t // 4 % 4 * 2) & 3
    if fmt == "FP3":
        x = x + 4 * (w[base + (4 + b // 4) * 1024 + lane * 16 + b % 4 * 4 + t % 4].int() >> (t // 4) & 1)
    at = base + (4096 if fmt == "FP2" else 6144) + lane * 16 + b * 2
    scale = (w[at].to(torch.int16) | w[at + 1].to(torch.int16) << 8).view(torch.float16).double()
    return (2 * x - (3 if fmt == "FP2" else 7)) * scale


def _exact_gemm(case, st):
    x = st["xq"].double() * st["xs"].double().repeat_interleave(32, 1)
    z = x @ _exact_weights(case, st["w"]).t()
    if st["bias"] is not None:
        z += st["bias"]
    act = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: z * torch.special.ndtr(z),
           "gelu_tanh": lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[case["act"]]
    z = act(z)
    return z if st["resid"] is None else z + st["resid"]


def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_rope if case["op"] == "rope" else _exact_attn if case["op"] == "attn" else _exact_gemm)(case, st)
