"""A serving step as a program runs it: sequences that share a prefix, each
request with its own adapters, through norm, projections, rotation with the
append, attention, output projection, a second norm with the residual, the MoE
layer, and a head with the log probabilities of drafted tokens."""

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R
import inputgen
from gpu_common import need_gpu, say
from moe_common import LayerSpec
from test_gpu_attention_layer import D, H, HK, HQ, batch_of, new_cache

pytestmark = pytest.mark.gpu
VOCAB, N_ADAPTERS, RANK = 777, 5, 16


def attention(seed, **kw):
    w = lambda m, r, c: inputgen.dense_weight(r, c, seed=100 * seed + m)  # noqa: E731
    return R.DeviceAttention.build(H, HQ, HK, D, w, rot_dim=16, in_norm=1 + 0.2 * inputgen.raw_normal(seed + 7, H), **kw)


def adapters(seed, scale=None):
    g = torch.Generator().manual_seed(seed)
    scale = (torch.rand(N_ADAPTERS, generator=g) if scale is None else torch.full((N_ADAPTERS,), scale)).cuda()
    return [R.DeviceLora((torch.randn(N_ADAPTERS, RANK, K, generator=g) * K ** -0.5).bfloat16().cuda(),
                         torch.randn(N_ADAPTERS, N, RANK, generator=g).bfloat16().cuda(), scale)
            for N, K in ((HQ * D, H), (HK * D, H), (HK * D, H), (H, HQ * D))]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# four sequences behind one prefix of 40 tokens: pages 0 and 1 are shared, the
# third page is each one's own
TABLE = [[0, 1, 2 + s, 6 + s] for s in range(4)]


def filled_cache(seed=0):
    c = new_cache(n_pages=12)
    g = torch.Generator().manual_seed(seed)
    for t in (c.k, c.v):
        t.copy_(torch.randn(t.shape, generator=g).half())
        for s in range(1, 4): # tokens 32 .. 39 are copies
            t[2 + s, :, :8] = t[2, :, :8]
    return c


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 1, 0, 4]])
def test_attention_half_is_its_entry_points(new):
    """run() against the calls it stands for, bit for bit, and against the
    half without the extras, which it must match where they say nothing."""
    need_gpu()
    T, layer, loras = sum(new), attention(1), adapters(2)
    ids = i32([(3 * t) % (N_ADAPTERS + 1) - 1 for t in range(T)])
    total = [40 + 5 * s + n for s, n in enumerate(new)]
    batch, pre = batch_of(new, total, i32(TABLE)), R.KVPrefix(i32([0, 4]), i32([40]), T, 40)
    x = torch.from_numpy(inputgen.raw_normal(3, (T, H))).cuda()
    caches = [filled_cache() for _ in range(4)]
    buf = R.AttentionBuffers(layer, caches[0], batch, prefix=pre, loras=loras)
    y = buf.run(layer, x, caches[0], batch, resid=x, prefix=pre, loras=loras, ids=ids).clone()

    b = R.AttentionBuffers(layer, caches[1], batch, prefix=pre, loras=loras)
    xn = torch.empty_like(x)
    R.add_rms_norm(x, layer.in_norm, layer.eps, None, None, xn, *b.x_act)
    if T <= 4:
        R.gemv_grouped(b._jobs(layer), b.ws_jobs)
    else:
        for W, o in ((layer.wq, b.q), (layer.wk, b.k), (layer.wv, b.v)):
            R.gemm(W, *b.x_act, T, o, ws=b.ws_gemm)
    R.lora(xn, ids, loras[:3], [o.view(T, -1) for o in (b.q, b.k, b.v)], ws=b.ws_lora)
    R.qk_norm_rope(b.q, b.k, b.v, caches[1], batch, b.q16, layer.inv_freq, eps=layer.eps)
    b.o.zero_()
    R.attn_shared(b.q16, caches[1], batch, pre, b.o, layer.scale, b.ws_attn)
    R.quantize_act(b.o.view(T, -1), *b.o_act)
    R.gemm(layer.wo, *b.o_act, T, b.y, resid=x, ws=b.ws_gemm)
    R.lora(b.o.view(T, -1), ids, loras[3:], [b.y], ws=b.ws_lora)
    assert torch.equal(y, b.y) and torch.equal(caches[0].k, caches[1].k)

    # adapters of factor zero, or for no one, change nothing; a prefix changes
    # the order of a softmax's sums, whose fp32 differences (2^-20) the
    # projection's 8-bit input may turn into a code more or less, 1 / 127 of a
    # block's largest value, for less than one value in a hundred: 1 / 1270
    same = R.AttentionBuffers(layer, caches[2], batch, prefix=pre).run(layer, x, caches[2], batch, resid=x, prefix=pre).clone()
    for kw in (dict(loras=adapters(2, 0.0), ids=ids), dict(loras=loras, ids=torch.full_like(ids, -1))):
        c = filled_cache()
        assert torch.equal(buf.run(layer, x, c, batch, resid=x, prefix=pre, **kw), same)
    alone = buf.run(layer, x, caches[3], batch, resid=x)
    assert float((alone - same).norm() / same.norm()) < 1e-3 and not torch.equal(y, same)


def test_input_norm_is_a_norm():
    """The half over a normed input without in_norm, whose codes differ by one
    where the two quantizers' scales differ by a step."""
    need_gpu()
    layer, plain = attention(4), attention(4)
    plain.in_norm = None
    batch = batch_of([5, 2], [5, 2], i32([[3, 1, 6, 0], [2, 7, 5, 4]]))
    x = torch.from_numpy(inputgen.raw_normal(5, (7, H))).cuda()
    xn = (x.double() / (x.double().square().mean(-1, keepdim=True) + layer.eps).sqrt() * layer.in_norm.double()).float()
    a, b = new_cache(), new_cache()
    y = R.AttentionBuffers(layer, a, batch).run(layer, x, a, batch, resid=x)
    z = R.AttentionBuffers(plain, b, batch).run(plain, xn, b, batch, resid=x)
    assert float((y - z).norm() / z.norm()) < 1e-3


class Model:
    def __init__(self):
        self.layers = [(attention(i), 1 + 0.1 * torch.from_numpy(inputgen.raw_normal(60 + i, H)).cuda(),
                        LayerSpec(i, H, 64, 8).build_device(), adapters(80 + i)) for i in range(2)]
        self.head = R.DeviceHead.build(VOCAB, H, inputgen.dense_weight(VOCAB, H, seed=9), fmt=R.FP4, norm=np.ones(H, np.float32))

    def buffers(self, caches, batch, pre):
        T, (a, _, moe, loras) = batch.n_tokens, self.layers[0]
        return (R.AttentionBuffers(a, caches[0], batch, prefix=pre, loras=loras), R.MoeBuffers(moe, T, 2),
                R.HeadBuffers(self.head, T, 4), torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda"))

    def step(self, bufs, x, caches, batch, pre, ids, tokens):
        """The residual stream in h; each half begins with a norm of it."""
        attn_buf, moe_buf, head_buf, h, xn = bufs
        h.copy_(x)
        for (attn, norm, moe, loras), cache in zip(self.layers, caches):
            a = attn_buf.run(attn, h, cache, batch, prefix=pre, loras=loras, ids=ids)
            R.add_rms_norm(h, norm, attn.eps, delta=a, out=h, y=xn)
            h.copy_(moe_buf.forward(moe, xn, resid=h))
        return head_buf.run(self.head, h, tokens)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [4, 2, 1, 3]])
def test_serving_steps(new):
    """Growing sequences, eager and as a captured graph replayed, with other
    adapters, tokens and lengths each time: the same bits; the verified tokens'
    log probabilities belong to the logits."""
    need_gpu()
    T, model = sum(new), Model()
    table = i32(TABLE)
    sets = []
    for _ in range(2):
        caches = [filled_cache(i) for i in range(2)]
        batch = batch_of(new, [40 + n for n in new], table)
        pre = R.KVPrefix(i32([0, 4]), i32([40]), T, 40)
        sets.append((caches, batch, pre, i32([0] * T), i32([0] * T), torch.zeros(T, H, device="cuda")))
    bufs = [model.buffers(*s[:3]) for s in sets]

    def one(i):
        caches, batch, pre, ids, tokens, x = sets[i]
        return model.step(bufs[i], x, caches, batch, pre, ids, tokens)

    one(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(0)
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        x = torch.randn(T, H, generator=g)
        ids, tokens = torch.randint(-1, N_ADAPTERS, (T,), generator=g), torch.randint(0, VOCAB, (T,), generator=g)
        for caches, batch, pre, *rest in sets:
            batch.kv_len.add_(2 if i else 0)
            pre.length.fill_(40 - 8 * (i == 2))
            for d, v in zip(rest, (ids, tokens, x)):
                d.copy_(v)
            for j, c in enumerate(caches):
                f = filled_cache(j)
                c.k.copy_(f.k), c.v.copy_(f.v)
        graph.replay()
        want = one(1)
        torch.cuda.synchronize()
        got = bufs[0][2].probs
        for name in ("logprob", "lse", "entropy", "rank", "top_index", "top_logprob"):
            assert torch.equal(getattr(got, name), getattr(want, name)), (i, name)
        for a, b in zip(sets[0][0], sets[1][0]):
            assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
        z = bufs[1][2].logits.double().cpu()
        lp = torch.log_softmax(z, -1)
        assert torch.isfinite(z).all()
        assert ((want.logprob.cpu().double() - lp.gather(1, tokens[:, None])[:, 0]).abs() <= 1e-5).all()
        assert torch.equal(want.top_index.cpu().long(), z.sort(dim=-1, descending=True, stable=True).indices[:, :4])
        assert ((want.entropy.cpu().double() + (lp.exp() * lp).sum(-1)).abs() <= 1e-5).all()


def test_two_calls_at_once():
    """On two streams, with a workspace each, the results are those of one
    after the other."""
    need_gpu()
    say("two streams")
    g = torch.Generator().manual_seed(5)
    T, rows, K, V = 96, 1024, 2048, 20000
    sides = []
    for side in range(2):
        b = R.DeviceKVCache(*(torch.randn((80, 2, 64, 128), generator=g).bfloat16().cuda() for _ in range(2)))
        table = torch.full((T, 2), -1, dtype=torch.int32)
        table[:, 0], table[:, 1] = side, torch.arange(T) % 70 + 5
        batch = R.KVBatch(i32(list(range(T + 1))), i32([64 + s % 64 + 1 for s in range(T)]), table.cuda(), T, 1)
        pre = R.KVPrefix(i32([0, T]), i32([64]), T, 64)
        lo = R.DeviceLora((torch.randn(9, 16, K, generator=g) * K ** -0.5).half().cuda(),
                          torch.randn(9, rows, 16, generator=g).half().cuda())
        x, z = torch.randn(T, K, generator=g).cuda(), torch.randn(T, V, generator=g).cuda()
        q = torch.randn((T, 8, 128), generator=g).bfloat16().cuda()
        d = dict(cache=b, batch=batch, pre=pre, lo=lo, x=x, z=z, q=q, ids=i32([(s * 5 + side) % 11 - 1 for s in range(T)]),
                 o=torch.empty(T, 8, 128, device="cuda"), y=torch.empty(T, rows, device="cuda"), h=torch.empty(T, K, device="cuda"),
                 p=R.LogprobBuffers(T, V, 20), tokens=i32([s * 77 for s in range(T)]))
        d["wa"] = torch.empty(R.attn_shared_workspace_bytes(b, batch, pre, 8), dtype=torch.uint8, device="cuda")
        d["wl"] = torch.empty(R.lora_workspace_bytes([lo], T), dtype=torch.uint8, device="cuda")
        sides.append(d)

    def run(d):
        R.add_rms_norm(d["x"], None, 1e-6, y=d["h"])
        R.lora(d["h"], d["ids"], [d["lo"]], [d["y"]], [None], d["wl"])
        R.attn_shared(d["q"], d["cache"], d["batch"], d["pre"], d["o"], 0.09, d["wa"])
        d["p"].run(d["z"], d["tokens"])

    def results(d):
        return [t.clone() for t in (d["h"], d["y"], d["o"], d["p"].logprob, d["p"].entropy, d["p"].top_index, d["p"].rank)]

    want = []
    for d in sides:
        run(d)
        torch.cuda.synchronize()
        want.append(results(d))
    streams = [torch.cuda.Stream() for _ in sides]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for d, s in zip(sides, streams):
            with torch.cuda.stream(s):
                run(d)
    torch.cuda.synchronize()
    for d, w in zip(sides, want):
        assert all(torch.equal(a, b) for a, b in zip(results(d), w))
