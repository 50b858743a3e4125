"""Host helpers that build an MoE layer in device memory and hold the
per-call buffers. Weights come from any provider of fp32 matrices; they are
quantized with the library's host encoder (rfx_quantize_matrix) and copied
to the GPU once."""

from __future__ import annotations

import ctypes
from concurrent.futures import ThreadPoolExecutor

import numpy as np

from . import (FP2, FP3, FP4, DeviceQMat, MoeLayerC, QMat, lib, moe_workspace_bytes,
               qmat_bytes, quantize_matrix)

GATE, UP, DOWN = 0, 1, 2


class DeviceMoeLayer:
    """Routed expert stacks (gate/up: inter x hidden, down: hidden x inter),
    an optional shared expert, and fp32 router weights/bias on the GPU."""

    def __init__(self, hidden, inter, n_experts, gate, up, down, sh=None, router_w=None,
                 router_b=None):
        self.hidden, self.inter, self.n_experts = hidden, inter, n_experts
        self.gate, self.up, self.down = gate, up, down
        self.sh = sh  # (gate, up, down) DeviceQMat or None
        self.router_w, self.router_b = router_w, router_b
        z = QMat(0, 0, 0, 0, None)
        c = MoeLayerC()
        c.hidden, c.inter, c.n_experts = hidden, inter, n_experts
        c.gate, c.up, c.down = gate.c, up.c, down.c
        if sh is not None:
            c.sh_gate, c.sh_up, c.sh_down = sh[0].c, sh[1].c, sh[2].c
        else:
            c.sh_gate = c.sh_up = c.sh_down = z
        c.router_w = router_w.data_ptr()
        c.router_b = router_b.data_ptr() if router_b is not None else None
        self.c = c

    def ref(self):
        return ctypes.byref(self.c)

    @classmethod
    def build(cls, hidden, inter, n_experts, weight_fn, router_w, router_b=None,
              fmt_gate=FP2, fmt_down=FP3, fmt_shared=FP4, shared=True, workers=8,
              device="cuda"):
        """weight_fn(expert, mat, rows, cols) -> fp32 [rows][cols]; mat is
        0 gate, 1 up, 2 down; expert == n_experts asks for the shared one."""
        import torch

        def stack(fmt, rows, cols, mat, count, first):
            nb = qmat_bytes(fmt, rows, cols)
            host = np.empty(count * nb, np.uint8)

            def one(e):
                W = weight_fn(first + e, mat, rows, cols)
                quantize_matrix(fmt, W, threads=1, out=host[e * nb:(e + 1) * nb])

            if count == 1:
                one(0)
            else:
                with ThreadPoolExecutor(workers) as ex:
                    list(ex.map(one, range(count)))
            return DeviceQMat(fmt, rows, cols, torch.from_numpy(host).to(device), count)

        gate = stack(fmt_gate, inter, hidden, GATE, n_experts, 0)
        up = stack(fmt_gate, inter, hidden, UP, n_experts, 0)
        down = stack(fmt_down, hidden, inter, DOWN, n_experts, 0)
        sh = None
        if shared:
            sh = (stack(fmt_shared, inter, hidden, GATE, 1, n_experts),
                  stack(fmt_shared, inter, hidden, UP, 1, n_experts),
                  stack(fmt_shared, hidden, inter, DOWN, 1, n_experts))
        rw = torch.from_numpy(np.ascontiguousarray(router_w, np.float32)).to(device)
        rb = None
        if router_b is not None:
            rb = torch.from_numpy(np.ascontiguousarray(router_b, np.float32)).to(device)
        return cls(hidden, inter, n_experts, gate, up, down, sh, rw, rb)

    def weight_bytes(self, experts, with_shared=True, with_router=True) -> int:
        """Packed bytes streamed for the given set of routed experts."""
        per = (qmat_bytes(self.gate.fmt, self.inter, self.hidden) * 2 +
               qmat_bytes(self.down.fmt, self.hidden, self.inter))
        n = per * len(set(int(e) for e in experts))
        if with_shared and self.sh is not None:
            n += (qmat_bytes(self.sh[0].fmt, self.inter, self.hidden) * 2 +
                  qmat_bytes(self.sh[2].fmt, self.hidden, self.inter))
        if with_router:
            n += self.n_experts * self.hidden * 4
        return n


def hot_experts_by_frequency(counts, n_hot):
    """The n_hot experts picked most often (ties to the lower id): the
    placement policy for a fixed budget of expert slots in HBM. counts: picks
    per expert from a warm-up run or the router's known bias."""
    counts = np.asarray(counts)
    order = np.lexsort((np.arange(len(counts)), -counts))
    return sorted(int(e) for e in order[:n_hot])


class PlacedMoeLayer(DeviceMoeLayer):
    """The experts of a DeviceMoeLayer placed by temperature: routed experts
    in `hot` stay in device memory (HBM), the others move to pinned host
    memory, which the kernels read directly over the host link; a device
    table of per-expert pointers ([gate e][up e][down e]) tells the kernels
    where each is (rfx_moe_layer.expert_data). The shared expert and the
    router stay in device memory."""

    def __init__(self, layer: DeviceMoeLayer, hot, device="cuda"):
        import torch
        E = layer.n_experts
        self.hot = sorted(set(int(e) for e in hot))
        hot_set = set(self.hot)
        self.cold = [e for e in range(E) if e not in hot_set]
        mats = (layer.gate, layer.up, layer.down)
        table = np.zeros((3, E), np.uint64)
        self.hot_data, self.cold_data = [], []
        for m, qm in enumerate(mats):
            nb = qmat_bytes(qm.fmt, qm.rows, qm.cols)
            hot_t = torch.empty(max(1, len(self.hot)) * nb, dtype=torch.uint8, device=device)
            cold_t = torch.empty(max(1, len(self.cold)) * nb, dtype=torch.uint8, pin_memory=True)
            for i, e in enumerate(self.hot):
                hot_t[i * nb:(i + 1) * nb].copy_(qm.data[e * nb:(e + 1) * nb])
                table[m, e] = hot_t.data_ptr() + i * nb
            for i, e in enumerate(self.cold):
                cold_t[i * nb:(i + 1) * nb].copy_(qm.data[e * nb:(e + 1) * nb])
                table[m, e] = cold_t.data_ptr() + i * nb
            self.hot_data.append(hot_t)
            self.cold_data.append(cold_t)
        torch.cuda.synchronize()
        self.table = torch.from_numpy(table.view(np.int64)).to(device)
        z = [DeviceQMat(qm.fmt, qm.rows, qm.cols, None, qm.count) for qm in mats]
        super().__init__(layer.hidden, layer.inter, E, z[0], z[1], z[2], layer.sh, layer.router_w, layer.router_b)
        self.c.expert_data = self.table.data_ptr()
        self.source = layer

    def hbm_bytes(self):
        """Packed routed-expert bytes held in device memory and in host memory."""
        per = sum(qmat_bytes(qm.fmt, qm.rows, qm.cols) for qm in (self.gate, self.up, self.down))
        return per * len(self.hot), per * len(self.cold)


class MoeBuffers:
    """Device buffers for one MoE decode call with q tokens, top-k."""

    def __init__(self, layer: DeviceMoeLayer, q: int, k: int, device="cuda"):
        import torch
        H, E = layer.hidden, layer.n_experts
        self.q, self.k = q, k
        self.topk_idx = torch.empty((q, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((q, k), dtype=torch.float32, device=device)
        self.pairs_sorted = torch.empty(q * k, dtype=torch.int32, device=device)
        self.expert_off = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.xq = torch.empty((q, H), dtype=torch.int8, device=device)
        self.xs = torch.empty((q, H // 32), dtype=torch.float32, device=device)
        self.xsum = torch.empty((q, H // 32), dtype=torch.int32, device=device)
        self.y = torch.empty((q, H), dtype=torch.float32, device=device)
        self.ws = torch.zeros(moe_workspace_bytes(layer, q, k), dtype=torch.uint8, device=device)

    def forward(self, layer: DeviceMoeLayer, x, resid=None, out=None, one_launch=False, stream=None):
        """The same as run(), through rfx_moe_forward: at q <= 4 the router
        launch computes the logits and every gate/up workgroup picks the top
        k itself (one_launch: the single-launch layer kernel for the page's
        formats instead)."""
        from . import moe_forward
        y = self.y if out is None else out
        moe_forward(layer, x, self.q, self.k, y, self.topk_idx, self.topk_w, self.pairs_sorted, self.expert_off,
                    self.xq, self.xs, self.xsum, self.ws, resid, one_launch, stream)
        return y

    def run(self, layer: DeviceMoeLayer, x, resid=None, out=None, stream=None):
        """route + FFN for x (device fp32 [q][hidden]); y = resid + MoE(x)
        lands in `out` (default self.y)."""
        from . import moe_ffn, moe_route_topk
        y = self.y if out is None else out
        moe_route_topk(layer, x, self.q, self.k, self.topk_idx, self.topk_w, self.pairs_sorted,
                       self.expert_off, self.xq, self.xs, self.xsum, self.ws, stream)
        moe_ffn(layer, self.q, self.k, self.xq, self.xs, self.xsum, self.topk_idx, self.topk_w,
                self.pairs_sorted, self.expert_off, y, self.ws, resid, stream)
        return y


Q_PROJ, K_PROJ, V_PROJ, O_PROJ = 0, 1, 2, 3


class DeviceAttention:
    """The attention half of a decoder layer on the GPU: packed query, key,
    value and output projections, optional per-head norm weights of queries
    and keys, rotary frequencies, and the mask's window and sinks."""

    def __init__(self, wq, wk, wv, wo, n_heads, n_kv_heads, head_dim, inv_freq, q_norm=None, k_norm=None, eps=1e-6,
                 interleaved=False, window=0, sinks=0, scale=None):
        if n_kv_heads < 1 or n_heads < 1 or n_heads % n_kv_heads:
            raise ValueError(f"{n_heads} heads over {n_kv_heads} kv heads")
        if window < 0 or sinks < 0 or not eps >= 0 or not (scale is None or scale > 0):
            raise ValueError(f"window {window}, sinks {sinks}, eps {eps}, scale {scale}")
        self.wq, self.wk, self.wv, self.wo = wq, wk, wv, wo
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        for W, rows, name in ((wq, n_heads, "wq"), (wk, n_kv_heads, "wk"), (wv, n_kv_heads, "wv")):
            if W.rows != rows * head_dim or W.cols != wq.cols:
                raise ValueError(f"{name}: {W.rows} x {W.cols}, {rows * head_dim} x {wq.cols} wanted")
        if wo.rows != wq.cols or wo.cols != n_heads * head_dim:
            raise ValueError(f"wo: {wo.rows} x {wo.cols}, {wq.cols} x {n_heads * head_dim} wanted")
        self.hidden = wq.cols
        self.inv_freq, self.q_norm, self.k_norm = inv_freq, q_norm, k_norm
        self.eps, self.interleaved, self.window, self.sinks = eps, interleaved, window, sinks
        self.scale = head_dim ** -0.5 if scale is None else scale

    @classmethod
    def build(cls, hidden, n_heads, n_kv_heads, head_dim, weight_fn, fmt=FP4, rot_dim=None, base=10000.0, q_norm=None,
              k_norm=None, device="cuda", **kw):
        """weight_fn(mat, rows, cols) -> fp32 [rows][cols]; mat is 0 query, 1
        key, 2 value, 3 output. q_norm, k_norm: fp32 [head_dim] or None."""
        import torch

        from . import rope_inv_freq

        def proj(mat, rows, cols):
            return DeviceQMat.from_host(fmt, rows, cols, quantize_matrix(fmt, weight_fn(mat, rows, cols)), device=device)

        def up(a):
            return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device)

        inv = torch.from_numpy(rope_inv_freq(head_dim if rot_dim is None else rot_dim, base)).to(device)
        return cls(proj(Q_PROJ, n_heads * head_dim, hidden), proj(K_PROJ, n_kv_heads * head_dim, hidden),
                   proj(V_PROJ, n_kv_heads * head_dim, hidden), proj(O_PROJ, hidden, n_heads * head_dim), n_heads,
                   n_kv_heads, head_dim, inv, up(q_norm), up(k_norm), **kw)


class AttentionBuffers:
    """Device buffers for attention calls over batches of this shape
    (n_tokens, max_q, sequences and page-table width as `batch` has them),
    for any layer with this one's formats and sizes."""

    def __init__(self, attn: DeviceAttention, cache, batch, device="cuda"):
        import torch

        from . import attn_workspace_bytes, gemm_workspace_bytes, gemv_grouped_workspace_bytes
        T, D, H = batch.n_tokens, attn.head_dim, attn.hidden
        O = attn.n_heads * D

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        def act(k):
            return empty(T, k, dtype=torch.int8), empty(T, k // 32), empty(T, k // 32, dtype=torch.int32)

        def zeros(n):
            return torch.zeros(n, dtype=torch.uint8, device=device) if n else None

        self.sizes = self._sizes(attn)
        self.x_act, self.o_act = act(H), act(O)
        self.q, self.k, self.v = (empty(T, h, D) for h in (attn.n_heads, attn.n_kv_heads, attn.n_kv_heads))
        self.q16 = empty(T, attn.n_heads, D, dtype=cache.dtype)
        with torch.inference_mode(False): # run clears o, inside such a mode or not
            self.o = empty(T, attn.n_heads, D)
        self.y = empty(T, H)
        mats = (attn.wq, attn.wk, attn.wv, attn.wo)
        self.ws_gemm = zeros(max(gemm_workspace_bytes(W, T) for W in mats))
        self.ws_attn = zeros(attn_workspace_bytes(cache, batch, attn.n_heads))
        self.ws_jobs = zeros(gemv_grouped_workspace_bytes(self._jobs(attn))) if T <= 4 else None

    @staticmethod
    def _sizes(attn):
        return attn.hidden, attn.n_heads, attn.n_kv_heads, attn.head_dim

    def _jobs(self, attn):
        """Decode's query, key and value projections, one launch."""
        from . import gemv_jobs
        return gemv_jobs([(W, self.q.shape[0], *self.x_act, y)
                          for W, y in zip((attn.wq, attn.wk, attn.wv), (self.q, self.k, self.v))])

    def run(self, attn: DeviceAttention, x, cache, batch, resid=None, out=None, stream=None):
        """Projections, norm, rotation and cache append, attention, output
        projection for x (device fp32 [n_tokens][hidden]); y = resid +
        Attention(x) lands in `out` (default self.y). Rows that attention
        leaves (of no sequence, of a skipped one, past max_q) have Attention(x)
        = 0. What does not fit these buffers is refused before anything is
        launched."""
        from . import _torch
        t, dev = _torch(), cache.index
        y = self.y if out is None else out
        jobs = self._jobs(attn) if batch.n_tokens <= 4 else None
        self._check(attn, x, cache, batch, resid, y, jobs)
        if dev >= 0 and t.current_device() != dev:
            with t.device_guard(dev):
                return self._run(attn, x, cache, batch, resid, y, jobs, stream)
        return self._run(attn, x, cache, batch, resid, y, jobs, stream)

    def _check(self, attn, x, cache, batch, resid, y, jobs):
        """The projections do not know how large their results' buffers are,
        and the append changes the cache: everything is looked at first."""
        from . import (_torch, _want, _want_vec, attn_workspace_bytes, gemm_workspace_bytes,
                       gemv_grouped_workspace_bytes)
        t, T, dev = _torch(), batch.n_tokens, cache.index
        if self.q.shape[0] != T:
            raise ValueError(f"buffers for {self.q.shape[0]} tokens, the batch has {T}")
        if self._sizes(attn) != self.sizes:
            raise ValueError(f"buffers for (hidden, heads, kv heads, head size) {self.sizes}, the layer has {self._sizes(attn)}")
        if (cache.n_kv_heads, cache.head_dim, cache.dtype) != (attn.n_kv_heads, attn.head_dim, self.q16.dtype):
            raise ValueError(f"cache of {cache.n_kv_heads} heads of {cache.head_dim} in {cache.dtype}, {attn.n_kv_heads} of "
                             f"{attn.head_dim} in {self.q16.dtype} wanted")
        places = self.q.get_device(), batch.index, attn.wq.index, attn.wk.index, attn.wv.index, attn.wo.index
        if places.count(dev) != 6:
            raise ValueError(f"buffers, batch, wq, wk, wv and wo on GPU {places}, the cache is on GPU {dev}")
        shape = T, attn.hidden
        _want(x, "x", t.f32, shape, dev)
        _want(y, "out", t.f32, shape, dev)
        if resid is not None:
            _want(resid, "resid", t.f32, shape, dev)
        _want_vec(attn.inv_freq, "inv_freq", t.f64, attn.inv_freq.numel(), dev)
        _want_vec(attn.q_norm, "q_norm", t.f32, attn.head_dim, dev)
        _want_vec(attn.k_norm, "k_norm", t.f32, attn.head_dim, dev)
        mats = (attn.wo,) if T <= 4 else (attn.wq, attn.wk, attn.wv, attn.wo)
        for name, ws, need in (("attention", self.ws_attn, attn_workspace_bytes(cache, batch, attn.n_heads)),
                               ("projections", self.ws_gemm, max(gemm_workspace_bytes(W, T) for W in mats)),
                               ("projections", self.ws_jobs, 0 if jobs is None else gemv_grouped_workspace_bytes(jobs))):
            if need > (0 if ws is None else ws.nbytes):
                raise ValueError(f"buffers have {0 if ws is None else ws.nbytes} bytes of workspace for the {name}, {need} wanted")

    def _run(self, attn, x, cache, batch, resid, y, jobs, stream):
        from . import _torch
        from . import attn as attention
        from . import gemm, gemv_grouped, qk_norm_rope, quantize_act
        T = batch.n_tokens
        quantize_act(x, *self.x_act, stream)
        if jobs is not None:
            gemv_grouped(jobs, self.ws_jobs, stream)
        else:
            for W, o in ((attn.wq, self.q), (attn.wk, self.k), (attn.wv, self.v)):
                gemm(W, *self.x_act, T, o, ws=self.ws_gemm, stream=stream)
        qk_norm_rope(self.q, self.k, self.v, cache, batch, self.q16, attn.inv_freq, attn.q_norm, attn.k_norm, attn.eps,
                     attn.interleaved, stream)
        # the rows that attention leaves must not carry an earlier call's on
        if stream is None:
            self.o.zero_()
        else:
            with _torch().on_stream(stream):
                self.o.zero_()
        attention(self.q16, cache, batch, self.o, attn.scale, attn.window, attn.sinks, self.ws_attn, stream)
        quantize_act(self.o.view(T, -1), *self.o_act, stream)
        gemm(attn.wo, *self.o_act, T, y, resid=resid, ws=self.ws_gemm, stream=stream)
        return y
