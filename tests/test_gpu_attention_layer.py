"""The attention half of a decoder layer as a program runs it (projections,
norm and rotation with the append, attention, output projection with the
residual) and a stack of attention and MoE layers: a prompt, then decoding
steps over the grown cache."""

import numpy as np
import pytest
import torch

import bit_block_quantized_amd as R
import inputgen
import oracle as O
from attn_common import rotate_exact
from gpu_common import need_gpu
from moe_common import LayerSpec

pytestmark = pytest.mark.gpu

H, HQ, HK, D = 256, 8, 2, 32


def build(seed=0, **kw):
    w = lambda m, r, c: inputgen.dense_weight(r, c, seed=100 * seed + m)  # noqa: E731
    norm = 1 + 0.2 * inputgen.raw_normal(seed + 50, (2, D))
    return R.DeviceAttention.build(H, HQ, HK, D, w, rot_dim=16, q_norm=norm[0], k_norm=norm[1], **kw), w, norm


def new_cache(n_pages=8, page=16):
    shape = (n_pages, HK, page, D)
    return R.DeviceKVCache(*(torch.full(shape, float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)))


def batch_of(new, total, table):
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    return R.KVBatch(off, torch.tensor(total, dtype=torch.int32, device="cuda"), table, int(sum(new)), max(new))


def rounded(x, fmt=None):
    """fp32 rows after the int8 activation quantizer, in 64 bits."""
    q, s = O.quantize_act(np.ascontiguousarray(x, np.float32))
    return q.astype(np.float64) * np.repeat(s.astype(np.float64), 32, axis=1)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_attention_half_stage_by_stage(T, window, sinks):
    """Each stage against its definition, fed by the stage before as the GPU
    computed it (so int8 codes on a border do not matter)."""
    need_gpu()
    layer, w, norm = build(window=window, sinks=sinks)
    cache = new_cache()
    table = torch.tensor([[3, 1, 6, 0]], dtype=torch.int32, device="cuda")
    batch = batch_of([T], [T], table)
    buf = R.AttentionBuffers(layer, cache, batch)
    x = inputgen.raw_normal(9, (T, H))
    xd = torch.from_numpy(x).cuda()
    y = buf.run(layer, xd, cache, batch, resid=xd).cpu().numpy()
    deq = [O.dequantize_matrix(4, O.quantize_matrix(4, w(m, *s))).astype(np.float64)
           for m, s in enumerate(((HQ * D, H), (HK * D, H), (HK * D, H), (H, HQ * D)))]
    xr = rounded(x)
    q, k, v = (t.cpu().numpy().reshape(T, -1) for t in (buf.q, buf.k, buf.v))
    for got, W in zip((q, k, v), deq):
        # block sums in fp32: 2^-20 of sum |w x| holds 10 blocks' roundings
        assert (np.abs(got - xr @ W.T) <= 2.0 ** -20 * (np.abs(xr) @ np.abs(W).T)).all()
    pos = torch.arange(T)
    ref, mag = rotate_exact(torch.from_numpy(q).view(T, HQ, D), torch.from_numpy(norm[0]), 1e-6, pos, layer.inv_freq.cpu(), False)
    q16 = buf.q16.cpu().double()
    assert ((q16 - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -15 * mag + 2.0 ** -25).all()
    page = table[0].cpu().long()[pos // 16]
    kk, vv = cache.k.cpu().double()[page, :, pos % 16], cache.v.cpu().double()[page, :, pos % 16]
    seen = pos[None] <= pos[:, None]
    if window:
        seen &= (pos[None] > pos[:, None] - window) | (pos[None] < sinks)
    o = buf.o.cpu().double()
    for h in range(HQ):
        s = (q16[:, h] @ kk[:, h // 4].t() * D ** -0.5).masked_fill(~seen, -np.inf)
        p = torch.softmax(s, -1)
        # scores below 30 over 32 elements: relative weights to 2^-14 (attn_bound's terms)
        assert ((o[:, h] - p @ vv[:, h // 4]).abs() <= 2.0 ** -14 * (p @ vv[:, h // 4].abs())).all()
    orr = rounded(buf.o.cpu().numpy().reshape(T, -1))
    assert (np.abs(y - x - orr @ deq[3].T) <= 2.0 ** -20 * (np.abs(orr) @ np.abs(deq[3]).T + np.abs(x))).all()


def test_stack_with_moe_prompt_then_decode():
    """Two layers of attention and MoE over two sequences: a prompt, a
    verification step of two tokens each, and single tokens. Runs, writes no
    NaN from the cache's empty slots, and the same calls give the same bits."""
    need_gpu()
    layers = [(build(i)[0], LayerSpec(i, H, 64, 8).build_device()) for i in range(2)]
    table = torch.tensor([[3, 1, 6, 0], [2, 7, 5, 4]], dtype=torch.int32, device="cuda")

    def decode():
        caches = [new_cache() for _ in layers]
        outs, total = [], [0, 0]
        for step, new in enumerate(([20, 13], [2, 2], [1, 1], [1, 1])):
            total = [t + n for t, n in zip(total, new)]
            batch = batch_of(new, total, table)
            x = torch.from_numpy(inputgen.raw_normal(step, (sum(new), H))).cuda()
            for (attn, moe), cache in zip(layers, caches):
                x = R.AttentionBuffers(attn, cache, batch).run(attn, x, cache, batch, resid=x).clone()
                x = R.MoeBuffers(moe, sum(new), 2).forward(moe, x, resid=x).clone()
            outs.append(x)
        torch.cuda.synchronize()
        return outs

    a, b = decode(), decode()
    for x, y in zip(a, b):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_layer_refuses_mismatched_projections():
    need_gpu()
    layer = build()[0]
    with pytest.raises(ValueError):
        R.DeviceAttention(layer.wq, layer.wq, layer.wv, layer.wo, HQ, HK, D, layer.inv_freq)
    with pytest.raises(ValueError):
        R.DeviceAttention(layer.wq, layer.wk, layer.wv, layer.wk, HQ, HK, D, layer.inv_freq)


@pytest.mark.parametrize("new", [[1, 1], [20, 13]])
def test_layers_share_buffers(new):
    """One set of buffers through two layers in turn, on a side stream: each
    gives what it gives with buffers of its own."""
    need_gpu()
    layers = [build(i)[0] for i in range(2)]
    table = torch.tensor([[3, 1, 6, 0], [2, 7, 5, 4]], dtype=torch.int32, device="cuda")
    batch = batch_of(new, new, table)
    x = torch.from_numpy(inputgen.raw_normal(3, (sum(new), H))).cuda()
    caches = [new_cache() for _ in range(4)]
    own = [R.AttentionBuffers(a, c, batch).run(a, x, c, batch).clone() for a, c in zip(layers, caches)]
    side = torch.cuda.Stream()
    shared = R.AttentionBuffers(layers[0], caches[2], batch)
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(x) for _ in layers]
    for a, c, y in zip(layers, caches[2:], out):
        shared.run(a, x, c, batch, out=y, stream=side)
    side.synchronize()
    assert not torch.equal(own[0], own[1])
    for y, want in zip(out, own):
        assert torch.equal(y, want)


def test_buffers_refuse_other_shapes():
    need_gpu()
    layer, cache = build()[0], new_cache()
    table = torch.tensor([[3, 1, 6, 0]], dtype=torch.int32, device="cuda")
    small, large = batch_of([3], [3], table), batch_of([5], [5], table)
    buf = R.AttentionBuffers(layer, cache, small)
    x = torch.zeros(5, H, device="cuda")
    for args, kw in (((x, cache, large), {}), ((x, cache, small), {}), ((x[:3, :32], cache, small), {}),
                     ((x[:3].double(), cache, small), {}), ((x[:3], cache, small), dict(out=x)),
                     ((x[:3], cache, small), dict(resid=x)), ((x[:3].cpu(), cache, small), {})):
        with pytest.raises(ValueError):
            buf.run(layer, *args, **kw)
    buf.run(layer, x[:3], cache, small)


@pytest.mark.parametrize("T,new", [(4, [1, 1]), (40, [20, 3])])
@pytest.mark.parametrize("how", ["current", "stream", "handle"])
def test_rows_of_no_sequence_get_the_residual_alone(T, new, how):
    """Padding rows, and rows past max_q, of a batch whose buffers held a full
    batch before: what attention leaves does not reach the result."""
    need_gpu()
    layer = build()[0]
    table = torch.tensor([[3, 1, 6, 0], [2, 7, 5, 4]], dtype=torch.int32, device="cuda")
    x = torch.from_numpy(inputgen.raw_normal(3, (T, H))).cuda()

    def batch(lead, new, max_q):
        off = torch.tensor(np.concatenate([[lead], lead + np.cumsum(new)]), dtype=torch.int32, device="cuda")
        return R.KVBatch(off, torch.tensor(new, dtype=torch.int32, device="cuda"), table, T, max_q)

    full, part = batch(0, [T // 2, T - T // 2], T), batch(1, new, T)
    cache = new_cache()
    buf = R.AttentionBuffers(layer, cache, full)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = {"current": None, "stream": side, "handle": side.cuda_stream}[how]
    out = torch.empty_like(x)
    live = torch.zeros(T, dtype=torch.bool)
    live[1:1 + sum(new)] = True
    for resid in (None, x):
        buf.run(layer, x, cache, full, stream=stream)
        buf.run(layer, x, cache, part, resid, out, stream)
        torch.cuda.synchronize()
        want = torch.zeros_like(x) if resid is None else x
        assert torch.equal(out[~live.cuda()], want[~live.cuda()])
        assert (out[live.cuda()] != want[live.cuda()]).any(1).all()
    short = batch(0, [T // 2, T - T // 2], 1)
    buf.run(layer, x, cache, full, stream=stream)
    buf.run(layer, x, cache, short, out=out, stream=stream)
    torch.cuda.synchronize()
    first = torch.zeros(T, dtype=torch.bool, device="cuda")
    first[[0, T // 2]] = True
    assert not out[~first].any() and out[first].any(1).all()


@pytest.mark.parametrize("new", [[1, 1], [20, 13]])
def test_captured_and_replayed(new):
    """The whole half captured once and replayed while the sequences grow,
    and while one of them has no rows, with eager calls between: every replay
    equals the eager result and leaves the same cache."""
    need_gpu()
    layer = build()[0]
    table = torch.tensor([[3, 1, 6, 0], [2, 7, 5, 4]], dtype=torch.int32, device="cuda")
    T = sum(new)
    batch = batch_of(new, new, table)
    x = torch.from_numpy(inputgen.raw_normal(3, (T, H))).cuda()
    caches = [R.DeviceKVCache(*(torch.zeros((8, HK, 16, D), dtype=torch.float16, device="cuda") for _ in range(2))) for _ in range(2)]
    bufs = [R.AttentionBuffers(layer, c, batch) for c in caches]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bufs[0].run(layer, x, caches[0], batch, resid=x)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        yg = bufs[0].run(layer, x, caches[0], batch, resid=x)
    off = batch.q_off.clone()
    for i in range(5):
        batch.kv_len.add_(3)
        batch.q_off.copy_(off)
        if i == 3: # the second sequence is away: its rows belong to none
            batch.q_off[2] = batch.q_off[1]
        x.copy_(torch.from_numpy(inputgen.raw_normal(30 + i, (T, H))))
        for c in caches:
            c.k.zero_(), c.v.zero_()
        ye = bufs[1].run(layer, x, caches[1], batch, resid=x)
        torch.cuda.synchronize()
        yg.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, ye), i
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v), i
        if i == 3:
            assert torch.equal(yg[new[0]:], x[new[0]:])
