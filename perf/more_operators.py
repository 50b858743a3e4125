"""Measured cases of what a serving step runs around the packed products, the
MoE layer and the paged attention: the residual's addition with an RMS norm
and 8-bit activations ("norm"), low-rank adapters of many requests beside a
shared projection ("lora"), attention of sequences that share a prefix
("shared"), and log probabilities of tokens from a head's logits ("logp").

run() computes the plain form (elementary torch operations in 32 bits, in 64
where a rounding decides) or, with `own` set, calls the library.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 2.0 ** -20  # an fp32 number, so that both sides add the same


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's residual stream before a decode step's projections: the
        # smallest call, where the launch itself counts
        dict(name="norm 1 token", op="norm", q=1, cols=4096, delta=True, weight=True, y=False, codes=True),
        # four verification positions before the router, which takes fp32
        dict(name="norm verify", op="norm", q=4, cols=7168, delta=True, weight=True, y=True, codes=False),
        # a prompt, fp32 for the adapters and codes for the projections
        dict(name="norm prompt", op="norm", q=4099, cols=7168, delta=True, weight=True, y=True, codes=True),
        # one token of one request, its query, key and value projections
        dict(name="lora 1 token", op="lora", type="bf16", tokens=1, runs=1, adapters=8, rank=16, cols=4096, rows=4096,
             kv_rows=1024, bare=False),
        # a serving batch of single tokens, every request its own adapter
        dict(name="lora 64 requests", op="lora", type="f16", tokens=64, runs=64, adapters=48, rank=64, cols=4096,
             rows=4096, kv_rows=0, bare=True),
        # prompts of several requests of different lengths, some with no
        # adapter
        dict(name="lora prompts", op="lora", type="bf16", tokens=4001, runs=7, adapters=12, rank=32, cols=4096, rows=4096,
             kv_rows=1024, bare=True),
        # a few answers to one short instruction
        dict(name="shared 4x1", op="shared", type="bf16", out="f32", groups=1, per_group=4, q_max=1, prefix=500, ctx=60,
             ragged=True, heads=32, kv_heads=8, dim=128, page=16),
        # four verification positions of the requests to two systems
        dict(name="shared verify 2x12x4", op="shared", type="f16", out="f32", groups=2, per_group=12, q_max=4, prefix=3001,
             ctx=300, ragged=True, heads=32, kv_heads=4, dim=128, page=64),
        # a serving batch behind one long document
        dict(name="shared 64x1 long", op="shared", type="bf16", out="same", groups=1, per_group=64, q_max=1, prefix=16384,
             ctx=700, ragged=True, heads=32, kv_heads=8, dim=128, page=64),
        # one sampled token's log probability with a few alternatives
        dict(name="logp 1 token", op="logp", type="f32", q=1, vocab=32000, top=5, masked=False),
        # verification of four positions of 16 sequences, half the vocabulary
        # excluded by a grammar
        dict(name="logp verify", op="logp", type="f32", q=64, vocab=131072, top=20, masked=True),
        # scoring of a prompt, 16-bit logits with many equal ones
        dict(name="logp prompt", op="logp", type="bf16", q=1021, vocab=100003, top=1, masked=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "lora", "shared", "logp"))
    if op == "norm":
        cols = 32 * _log(rng, 4, 512)
        y = rng.random() < 0.5
        return dict(op="norm", q=_log(rng, 1, min(8192, 29_000_000 // cols)), cols=cols, delta=rng.random() < 0.8,
                    weight=rng.random() < 0.8, y=y, codes=not y or rng.random() < 0.5)
    if op == "lora":
        cols, rows, rank = 32 * _log(rng, 8, 224), _log(rng, 33, 7168), 8 * _log(rng, 1, 16)
        tokens = _log(rng, 1, min(4001, 16_000_000 // max(cols, rows)))
        return dict(op="lora", type=rng.choice(("bf16", "f16")), tokens=tokens, runs=rng.randint(1, min(tokens, 64)),
                    adapters=_log(rng, 1, 48), rank=rank, cols=cols, rows=rows,
                    kv_rows=rng.choice((0, max(1, rows // 4))), bare=rng.random() < 0.5)
    if op == "shared":
        kv_heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 80, 128, 128, 256))
        heads = kv_heads * rng.choice((1, 2, 4, 8))
        groups = rng.randint(1, 3)
        per_group = _log(rng, 2, 64 // groups)
        return dict(op="shared", type=rng.choice(("bf16", "f16")), out=rng.choice(("f32", "same")), groups=groups,
                    per_group=per_group, q_max=rng.randint(1, 4), prefix=_log(rng, 30, 16384 // groups),
                    ctx=_log(rng, 1, 700), ragged=rng.random() < 0.7, heads=heads, kv_heads=kv_heads, dim=dim,
                    page=rng.choice((1, 8, 16, 32, 64, 256)))
    vocab = _log(rng, 500, 150000)
    return dict(op="logp", type=rng.choice(("f32", "f32", "bf16", "f16")), q=_log(rng, 1, min(2048, 50_000_000 // vocab)),
                vocab=vocab, top=rng.choice((0, 1, 5, 20, 64)), masked=rng.random() < 0.3)


def _ids(case):
    """The adapter of each token: requests one after the other, each a run of
    tokens with one adapter, every fourth request without one where the case
    says so."""
    rng = random.Random("%d %d %d" % (case["tokens"], case["runs"], case["adapters"]))
    cut = [0] + sorted(rng.sample(range(1, case["tokens"]), case["runs"] - 1)) + [case["tokens"]]
    order = list(range(case["adapters"]))
    rng.shuffle(order)
    ids = []
    for i in range(case["runs"]):
        a = -1 if case["bare"] and i % 4 == 3 else order[i % len(order)]
        ids += [a] * (cut[i + 1] - cut[i])
    return ids


def _lengths(case):
    """(prefix of each group, [(new tokens, cached tokens with the new ones)]
    of each sequence): the first group and sequence at the case's bounds, the
    others, where the case is ragged, anywhere below, every ninth sequence
    with no new token."""
    rng = random.Random("%d %d %d %d" % (case["groups"], case["per_group"], case["prefix"], case["ctx"]))
    prefix, seqs = [], []
    for g in range(case["groups"]):
        p = case["prefix"] if not g or not case["ragged"] else rng.randint(case["prefix"] // 2, case["prefix"])
        prefix.append(p)
        for s in range(case["per_group"]):
            n, c = case["q_max"], case["ctx"]
            if case["ragged"] and (g or s):
                n = 0 if s % 9 == 8 else rng.randint(1, n)
                c = rng.randint(0, c)
            seqs.append((n, p + c + n))
    return prefix, seqs


# ----------------------------------------------------------------- inputs

def _normal(gen, shape, sigma=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(sigma).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _prepare_norm(st, case, gen):
    q, K = case["q"], case["cols"]
    # a residual stream has a few columns far larger than the rest
    x = _normal(gen, (q, K))
    x[:, :: max(1, K // 5)] *= 20
    st["x"] = x
    st["delta"] = _normal(gen, (q, K), 0.3) if case["delta"] else None
    st["w"] = _normal(gen, (K,), 0.2).add_(1) if case["weight"] else None
    st["sum"] = _empty(q, K) if case["delta"] else None
    st["y"] = _empty(q, K) if case["y"] else None
    codes = case["codes"]
    st["xq"] = _empty(q, K, dtype=torch.int8) if codes else None
    st["xs"] = _empty(q, K // 32) if codes else None
    st["xsum"] = _empty(q, K // 32, dtype=torch.int32) if codes else None


def _prepare_lora(st, case, gen):
    T, K, r, n, t = case["tokens"], case["cols"], case["rank"], case["adapters"], TYPES[case["type"]]
    rows = [case["rows"]] + [case["kv_rows"]] * 2 * (case["kv_rows"] > 0)
    st["x"], st["ids"] = _normal(gen, (T, K)), _i32(_ids(case))
    # every adapter's alpha / rank
    st["scale"] = torch.rand(n, generator=gen, device=DEV) * 1.5 + 0.5
    st["a"] = [_normal(gen, (n, r, K), K ** -0.5, t) for _ in rows]
    st["b"] = [_normal(gen, (n, N, r), r ** -0.5, t) for N in rows]
    st["resid"] = [_normal(gen, (T, N)) for N in rows] # the shared projection's result
    st["y"] = [_empty(T, N) for N in rows]
    if own:
        R = st["R"]
        st["lora"] = [R.DeviceLora(a, b, st["scale"]) for a, b in zip(st["a"], st["b"])]
        st["ws"] = _empty(R.lora_workspace_bytes(st["lora"], T), dtype=torch.uint8)


def _prepare_shared(st, case, gen):
    prefix, seqs = _lengths(case)
    page, D, t = case["page"], case["dim"], TYPES[case["type"]]
    shared = [p // page for p in prefix] # whole pages that a group's tables have in common
    own_pages = [-(-total // page) - shared[s // case["per_group"]] for s, (_, total) in enumerate(seqs)]
    n_pages = sum(shared) + sum(own_pages) + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    width = max(-(-total // page) for _, total in seqs)
    table = torch.zeros((len(seqs), width), dtype=torch.int32, device=DEV)
    first, at = [], 0
    for n in shared:
        first.append(at)
        at += n
    for s, n in enumerate(own_pages):
        g = s // case["per_group"]
        table[s, :shared[g]] = order[first[g]:first[g] + shared[g]]
        table[s, shared[g]:shared[g] + n] = order[at:at + n]
        at += n
    off = [0]
    for n, _ in seqs:
        off.append(off[-1] + n)
    shape = (n_pages, case["kv_heads"], page, D)
    st["k_cache"], st["v_cache"] = _normal(gen, shape, dtype=t), _normal(gen, shape, dtype=t)
    # what is left of a prefix behind its last whole page is each sequence's
    # own copy of the same tokens
    for g, p in enumerate(prefix):
        lo, hi = g * case["per_group"], (g + 1) * case["per_group"]
        if p % page:
            ids = table[lo:hi, p // page].long()
            for c in (st["k_cache"], st["v_cache"]):
                c[ids, :, :p % page] = c[ids[0], :, :p % page]
    st["table"], st["q_off"], st["kv_len"] = table, _i32(off), _i32([c for _, c in seqs])
    st["tokens"] = off[-1]
    st["q"] = _normal(gen, (off[-1], case["heads"], D), dtype=t)
    st["scale"] = 1 / math.sqrt(D)
    st["out"] = _empty(off[-1], case["heads"], D, dtype=torch.float32 if case["out"] == "f32" else t)
    if own:
        R = st["R"]
        per = case["per_group"]
        st["cache"] = R.DeviceKVCache(st["k_cache"], st["v_cache"])
        st["batch"] = R.KVBatch(st["q_off"], st["kv_len"], table, off[-1], case["q_max"])
        st["prefix"] = R.KVPrefix(_i32([g * per for g in range(case["groups"] + 1)]), _i32(prefix),
                                  max(off[(g + 1) * per] - off[g * per] for g in range(case["groups"])), max(prefix))
        n = R.attn_shared_workspace_bytes(st["cache"], st["batch"], st["prefix"], case["heads"])
        st["ws"] = _empty(n, dtype=torch.uint8) if n else None


def _prepare_logp(st, case, gen):
    q, V, k = case["q"], case["vocab"], case["top"]
    z = _normal(gen, (q, V), 2.5)
    # a few likely tokens in every row, as a trained head has them
    likely = torch.randint(0, V, (q, 12), generator=gen, device=DEV)
    z.scatter_add_(1, likely, torch.rand((q, 12), generator=gen, device=DEV) * 14)
    st["tokens"] = likely[:, 0].to(torch.int32)
    if case["masked"]:
        out = torch.rand((q, V), generator=gen, device=DEV) < 0.5
        out.scatter_(1, likely[:, :1], False)
        z.masked_fill_(out, -math.inf)
    st["z"] = z.to(TYPES[case["type"]])
    if own:
        st["buf"] = st["R"].LogprobBuffers(q, V, k)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)
    st = dict(case=dict(case))
    if own:
        import bit_block_quantized_amd as R
        st["R"] = R
    {"norm": _prepare_norm, "lora": _prepare_lora, "shared": _prepare_shared, "logp": _prepare_logp}[case["op"]](st, case, gen)
    return st


# ------------------------------------------------------------- plain forms

def _plain_norm(st):
    q, K = st["x"].shape
    out = {}
    h = st["x"]
    if st["delta"] is not None:
        h = out["sum"] = h + st["delta"]
    # in 64 bits, so that y is the nearest fp32 number: it decides the codes
    h = h.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    if st["w"] is not None:
        y = y * st["w"].double()
    y = y.float()
    if st["y"] is not None:
        out["y"] = y
    if st["xq"] is not None:
        y = y.view(q, K // 32, 32)
        s = y.abs().amax(-1) / 127
        c = torch.round(y / torch.where(s == 0, 1.0, s)[..., None]).clamp(-127, 127)
        out["codes"], out["scales"] = c.view(q, K).to(torch.int8), s # whole numbers, equal on both sides
        out["code_sums"] = c.sum(-1).to(torch.int32)
    return out


def _plain_lora(st):
    """All adapters' first factors as one product, what is not a token's own
    set to zero, all second factors as one product."""
    case = st["case"]
    T, n, r, K = case["tokens"], case["adapters"], case["rank"], case["cols"]
    mine = st["ids"][:, None] == torch.arange(n, device=DEV)
    factor = torch.where(mine, st["scale"], 0.0)[..., None]
    out = []
    for a, b, resid in zip(st["a"], st["b"], st["resid"]):
        v = (st["x"] @ a.float().view(n * r, K).t()).view(T, n, r) * factor
        out.append(resid + v.view(T, n * r) @ b.float().transpose(1, 2).reshape(n * r, -1))
    return out


def _plain_shared(st):
    """Every sequence over all its keys, padded to the longest."""
    case = st["case"]
    n, mq, page = st["table"].shape[0], case["q_max"], case["page"]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G, L = Hq // Hk, st["table"].shape[1] * page
    ids = st["table"].long()
    k = st["k_cache"][ids].transpose(1, 2).reshape(n, Hk, L, D).float()
    v = st["v_cache"][ids].transpose(1, 2).reshape(n, Hk, L, D).float()
    new = st["q_off"][1:] - st["q_off"][:-1]
    i = torch.arange(mq, device=DEV)
    row = (st["q_off"][:-1, None] + i).clamp_(max=st["tokens"] - 1).long()
    q = st["q"][row].float().reshape(n, mq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hk, mq * G, D)
    pos = (st["kv_len"] - new)[:, None] + i
    seen = torch.arange(L, device=DEV) <= pos[..., None]
    score = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(n, Hk, mq, G, L)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, Hk, mq * G, L) @ v).view(n, Hk, mq, G, D) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(n, mq, Hq, D)
    t = torch.arange(st["tokens"], device=DEV, dtype=torch.int32)
    s = torch.searchsorted(st["q_off"][1:].contiguous(), t, right=True)
    st["out"].copy_(o[s, (t - st["q_off"][s]).long()])
    return st["out"]


def _plain_logp(st):
    z, k = st["z"].float(), st["case"]["top"]
    token = st["tokens"].long()[:, None]
    top = z.amax(-1, keepdim=True)
    d = z - top
    e = d.exp()
    total = e.sum(-1, keepdim=True, dtype=torch.float64) # long sums
    lse = top + total.log()
    mean = torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True, dtype=torch.float64) / total
    mine = z.gather(1, token)
    out = dict(logprob=(mine - lse).float().squeeze(1), lse=lse.float().squeeze(1),
               entropy=(total.log() - mean).float().squeeze(1), rank=(z > mine).sum(-1).to(torch.int32))
    if k:
        # a key that is larger for a larger value and, at equal ones, for the lower index
        bits = z.view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = (order << 32) + (0x7fffffff - torch.arange(z.shape[1], device=DEV))
        i = 0x7fffffff - (key.topk(k, -1).values & 0xffffffff)
        out["top_index"] = i.to(torch.int32)
        out["top_logprob"] = (z.gather(1, i) - lse).float()
    return out


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "lora": _plain_lora, "shared": _plain_shared, "logp": _plain_logp}[op](st)
    R = st["R"]
    if op == "norm":
        R.add_rms_norm(st["x"], st["w"], EPS, delta=st["delta"], out=st["sum"], y=st["y"], xq=st["xq"], xs=st["xs"],
                       xsum=st["xsum"])
        named = dict(sum=st["sum"], y=st["y"], codes=st["xq"], scales=st["xs"], code_sums=st["xsum"])
        return {k: v for k, v in named.items() if v is not None}
    if op == "lora":
        R.lora(st["x"], st["ids"], st["lora"], st["y"], st["resid"], st["ws"])
        return st["y"]
    if op == "shared":
        R.attn_shared(st["q"], st["cache"], st["batch"], st["prefix"], st["out"], st["scale"], st["ws"])
        return st["out"]
    b = st["buf"].run(st["z"], st["tokens"])
    out = dict(logprob=b.logprob, lse=b.lse, entropy=b.entropy, rank=b.rank)
    if st["case"]["top"]:
        out["top_index"], out["top_logprob"] = b.top_index, b.top_logprob
    return out


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        n = case["q"] * case["cols"]
        each = 4 + 8 * case["delta"] + 4 * case["y"] + (1.25 if case["codes"] else 0)
        return dict(bytes=int(n * each) + 4 * case["cols"] * case["weight"], flops=8 * n)
    if case["op"] == "lora":
        ids = _ids(case)
        rows = case["rows"] + 2 * case["kv_rows"]
        K, r, T, mats = case["cols"], case["rank"], case["tokens"], 1 + 2 * (case["kv_rows"] > 0)
        used, on = len(set(ids) - {-1}), sum(i >= 0 for i in ids)
        return dict(bytes=4 * T * K + 2 * used * r * (mats * K + rows) + 8 * T * rows, flops=2 * on * r * (mats * K + rows))
    if case["op"] == "shared":
        prefix, seqs = _lengths(case)
        Hq, Hk, D, T = case["heads"], case["kv_heads"], case["dim"], sum(n for n, _ in seqs)
        keys, pairs = sum(prefix), 0
        for s, (n, total) in enumerate(seqs):
            if n:
                keys += total - prefix[s // case["per_group"]]
                pairs += sum(range(total - n + 1, total + 1))
        wide = 4 if case["out"] == "f32" else 2
        return dict(bytes=4 * keys * Hk * D + T * Hq * D * (2 + wide), flops=4 * pairs * Hq * D)
    n = case["q"] * case["vocab"]
    return dict(bytes=n * TYPES[case["type"]].itemsize + case["q"] * (20 + 8 * case["top"]), flops=6 * n)


# ------------------------------------------------------- 64-bit definitions

def _exact_norm(case, st):
    out = {}
    h = st["x"].double()
    if case["delta"]:
        out["sum"] = h + st["delta"].double()
        h = out["sum"].float().double() # the stream is held in fp32
    w = torch.ones_like(h[0]) if st["w"] is None else st["w"].double()
    size = torch.linalg.vector_norm(h, dim=-1, keepdim=True) / math.sqrt(case["cols"])
    y = w * (h / torch.hypot(size, torch.full_like(size, math.sqrt(EPS))))
    if case["y"]:
        out["y"] = y
    if case["codes"]:
        # the codes are those of the fp32 numbers next to y
        b = y.float().unflatten(-1, (-1, 32))
        s = torch.linalg.vector_norm(b, math.inf, dim=-1) / 127
        # a quotient rounds to fp32 before it rounds to a whole number
        c = (b.double() / torch.where(s == 0, 1.0, s).double()[..., None]).float().double().round().clamp(-127, 127)
        out["codes"], out["scales"], out["code_sums"] = c.flatten(-2).to(torch.int8), s.double(), c.sum(-1).to(torch.int32)
    return out


def _exact_lora(case, st):
    out = [r.double() for r in st["resid"]]
    ids = st["ids"].tolist()
    x = st["x"].double()
    for a in sorted(set(ids) - {-1}):
        rows = torch.tensor([t for t, i in enumerate(ids) if i == a], device=DEV)
        for y, p, q in zip(out, st["a"], st["b"]):
            y[rows] += float(st["scale"][a]) * ((x[rows] @ p[a].double().t()) @ q[a].double().t())
    return out


def _exact_shared(case, st):
    _, seqs = _lengths(case)
    Hq, Hk, page = case["heads"], case["kv_heads"], case["page"]
    G = Hq // Hk
    out = torch.zeros((st["tokens"], Hq, case["dim"]), dtype=torch.float64, device=DEV)
    at = 0
    for s, (n, total) in enumerate(seqs):
        if n:
            ids = st["table"][s, :-(-total // page)].long()
            hidden = torch.arange(total, device=DEV)[None] > torch.arange(total - n, total, device=DEV)[:, None]
            for h in range(Hk):
                k = st["k_cache"][ids, h].double().flatten(0, 1)[:total]
                v = st["v_cache"][ids, h].double().flatten(0, 1)[:total]
                q = st["q"][at:at + n, h * G:(h + 1) * G].double().transpose(0, 1)
                z = (q @ k.t() * st["scale"]).masked_fill(hidden, -math.inf)
                out[at:at + n, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ v).transpose(0, 1)
        at += n
    return out


def _exact_logp(case, st):
    rows = []
    for z, token in zip(st["z"].split(64), st["tokens"].long().split(64)): # a few rows at a time
        z = z.double()
        log_p = z - torch.logsumexp(z, -1, keepdim=True)
        mine = z.gather(1, token[:, None])
        r = dict(logprob=log_p.gather(1, token[:, None])[:, 0], lse=torch.logsumexp(z, -1),
                 entropy=torch.special.entr(log_p.exp()).sum(-1), rank=(z > mine).sum(-1).to(torch.int32))
        if case["top"]:
            best = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
            r["top_index"], r["top_logprob"] = best.to(torch.int32), log_p.gather(1, best)
        rows.append(r)
    return {k: torch.cat([r[k] for r in rows]) for k in rows[0]}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "shared": _exact_shared, "logp": _exact_logp}[case["op"]](case, st)
