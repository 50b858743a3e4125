"""rfx_lora_apply against its definition in 64 bits: any order of adapters
among the tokens, tokens without one, ranks and rows that end inside tiles,
several matrices, results in place."""

import pytest
import torch

import bit_block_quantized_amd as R
from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    def __init__(self, T, K, rank, rows, adapters, kind, ids=None, scale=True, resid=True, seed=0):
        need_gpu()
        say(f"lora T={T} K={K} rank={rank} rows={rows} adapters={adapters} {kind}")
        g = torch.Generator().manual_seed(seed + T + K + rank)
        t = TYPES[kind]
        self.kind, self.K, self.rank = kind, K, rank
        self.x = torch.randn(T, K, generator=g) * 10.0 ** torch.linspace(-3, 2, T)[:, None]
        self.ids = torch.randint(-1, adapters + 1, (T,), generator=g) if ids is None else torch.tensor(ids)
        self.a = [(torch.randn(adapters, rank, K, generator=g) * K ** -0.5).to(t) for _ in rows]
        self.b = [torch.randn(adapters, N, rank, generator=g).to(t) for N in rows]
        self.scale = torch.rand(adapters, generator=g) * 2 - 0.5 if scale else None
        self.resid = [torch.randn(T, N, generator=g) if resid else None for N in rows]
        self.rows = rows

    def device(self):
        s = None if self.scale is None else self.scale.cuda()
        self.loras = [R.DeviceLora(a.cuda(), b.cuda(), s) for a, b in zip(self.a, self.b)]
        n = R.lora_workspace_bytes(self.loras, len(self.x))
        self.ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda") # NaN: it needs no initialisation
        self.ys = [torch.full((len(self.x), N), 7.0, device="cuda") for N in self.rows]
        return self.loras

    def run(self):
        self.device()
        R.lora(self.x.cuda(), self.ids.to(torch.int32).cuda(), self.loras, self.ys,
               [None if r is None else r.cuda() for r in self.resid], self.ws)
        return [y.cpu() for y in self.ys]

    def exact(self):
        """(y, bound) per matrix. A x is a sum of cols products, each of up to
        three terms, B (A x) of rank such products: fp32 sums in any order are
        off by at most a half step of 2^-24 of the sum of magnitudes per
        addition (and a few for the scale and the split). fp16's two terms
        leave 2^-22 of an operand (8 more half steps each) and 2^-32 of x
        below its subnormals."""
        step = 2.0 ** -24
        extra = 8 if self.kind == "f16" else 0
        for a, b, resid in zip(self.a, self.b, self.resid):
            T, N = len(self.x), b.shape[1]
            y = torch.zeros(T, N, dtype=torch.float64) if resid is None else resid.double()
            tol = step * y.abs() + 2.0 ** -140
            for ad in range(len(a)):
                on = (self.ids == ad).nonzero()[:, 0]
                if not len(on):
                    continue
                x, A, B = self.x[on].double(), a[ad].double(), b[ad].double()
                c = 1.0 if self.scale is None else float(self.scale[ad])
                v, mag = x @ A.t(), x.abs() @ A.abs().t()
                dv = (3 * self.K + 24 + extra) * step * mag
                if extra:
                    dv += 2.0 ** -32 * A.abs().sum(1)
                d, dm = c * (v @ B.t()), abs(c) * (v.abs() @ B.abs().t())
                y[on] += d
                tol[on] += abs(c) * (dv @ B.abs().t()) + (3 * self.rank + 8 + extra) * step * dm + 2 * step * d.abs()
            yield y, tol

    def check(self):
        for i, (got, (y, tol)) in enumerate(zip(self.run(), self.exact())):
            bad = ~((got.double() - y).abs() <= tol)
            assert not bad.any(), f"matrix {i}: {int(bad.sum())} outside, at {bad.nonzero()[0].tolist()}"
            # far inside: additions' errors have no common sign
            norm = float((got.double() - y).norm() / y.norm().clamp(min=1e-30))
            assert norm <= 2.0 ** -24 * (3 * self.K + 3 * self.rank + 64) ** 0.5 * 2, norm
        return self


SIZES = [(1, 32, 8, [1], 1), (1, 4096, 16, [4096, 1024, 1024], 4), (2, 64, 16, [5, 3], 3), (15, 96, 24, [63], 5),
         (16, 1056, 40, [257, 16, 30, 7], 3), (17, 4096, 64, [1000], 20), (33, 288, 128, [100, 60], 2),
         (64, 2048, 64, [512], 48), (130, 160, 8, [48], 50), (257, 512, 32, [300, 20], 9), (300, 96, 128, [70, 64, 5, 9], 30),
         (1000, 640, 16, [130], 4), (600, 1024, 56, [1026], 1)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_sizes(case, kind):
    Case(*SIZES[case], kind, scale=case % 3 != 0, resid=case % 4 != 1).check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T", [5, 40, 300])
def test_orders_of_adapters(T, kind):
    n = 6
    for name, ids in (("one", [3] * T), ("none", [-1] * T), ("past the last", [n, 2 ** 31 - 1, -2 ** 31] * T),
                      ("alternating", list(range(n)) * T), ("runs", sorted(list(range(-1, n)) * T)[::n]),
                      ("last alone", [-1] * (T - 1) + [5])):
        say(name)
        Case(T, 224, 16, [90, 33], n, kind, ids=ids[:T]).check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T", [3, 20, 400])
def test_in_place_and_strided(T, kind):
    c = Case(T, 320, 32, [96, 50], 3, kind)
    want = c.run()
    wide = torch.full((T, 512), float("nan"), device="cuda")
    wide[:, 64:384] = c.x.cuda()
    ids = c.ids.to(torch.int32).cuda()
    ys = [r.cuda() for r in c.resid]
    R.lora(wide[:, 64:384], ids, c.loras, ys, ws=c.ws)
    for y, w in zip(ys, want):
        assert torch.equal(y.cpu(), w)
    # one matrix at a time
    for m, w, r in zip(c.loras, want, c.resid):
        y = r.cuda()
        R.lora(wide[:, 64:384], ids, [m], [y], ws=c.ws)
        tol = (3 * 320 + 3 * 32 + 64) * 2.0 ** -23 * 200 # of |x| up to 100 sqrt(320)
        assert ((y.cpu() - w).abs() <= tol).all()
    # results that start anywhere
    flat = torch.zeros(T * 96 + 1, device="cuda")
    y = flat[1:].view(T, 96)
    R.lora(wide[:, 64:384], ids, c.loras[:1], [y], [c.resid[0].cuda()], c.ws)
    assert ((y.cpu() - want[0]).abs() <= tol).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_token_keeps_its_infinities(kind):
    c = Case(20, 128, 16, [40], 2, kind, ids=[0, 1] * 10)
    want = c.run()[0]
    c.x[4, 7], c.x[9, 100] = float("nan"), float("inf")
    got = c.run()[0]
    rest = [t for t in range(20) if t not in (4, 9)]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[9]).any()


def test_large_and_small_values():
    for kind in TYPES:
        for factor in (1e-12, 1e-4, 5e3):
            c = Case(18, 256, 16, [64], 3, kind, resid=False)
            c.x *= factor / c.x.abs().amax() * 100
            for got, (y, tol) in zip(c.run(), c.exact()):
                assert ((got.double() - y).abs() <= tol).all(), (kind, factor)


def test_no_tokens():
    c = Case(1, 64, 8, [16], 2, "bf16")
    c.device()
    R.lora(torch.zeros(0, 64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), c.loras,
           [torch.zeros(0, 16, device="cuda")])


@pytest.mark.parametrize("T", [4, 50, 300])
def test_captured_with_other_ids(T):
    """Ids, inputs and results change between replays; two runs are equal."""
    torch = need_gpu()
    c = Case(T, 512, 24, [200, 64], 7, "bf16")
    c.device()
    x, ids = c.x.cuda(), c.ids.to(torch.int32).cuda()
    resid = [r.cuda() for r in c.resid]
    R.lora(x, ids, c.loras, c.ys, resid, c.ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.lora(x, ids, c.loras, c.ys, resid, c.ws)
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        c.ids = torch.randint(-1, 8, (T,), generator=gen)
        c.x = torch.randn(T, 512, generator=gen)
        ids.copy_(c.ids)
        x.copy_(c.x)
        g.replay()
        torch.cuda.synchronize()
        for got, (y, tol) in zip(c.ys, c.exact()):
            assert ((got.cpu().double() - y).abs() <= tol).all()
        again = [torch.empty_like(y) for y in c.ys]
        R.lora(x, ids, c.loras, again, resid, c.ws)
        assert all(torch.equal(p, q) for p, q in zip(again, c.ys))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows", [[7001], [4096, 4100], [64, 7168]])
def test_many_tokens_and_rows(rows, kind):
    """So many that a workgroup takes rows twice, ends inside its second turn
    or has none."""
    Case(700, 64, 24, rows, 5, kind).check()
    Case(700, 64, 24, rows, 5, kind, ids=[0] * 40 + [-1] * 100 + [4] * 300 + [7] * 60 + [2] * 200, resid=False).check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,K,rank,rows", [(4, 96, 16, [50]), (20, 512, 8, [70, 33]), (64, 4096, 64, [512]), (130, 256, 40, [64, 64, 64]),
                                           (200, 1024, 128, [100, 40]), (300, 2048, 32, [96, 50]), (700, 64, 24, [4100])])
def test_an_adapter_keeps_its_infinities(T, K, rank, rows, kind):
    """Infinities and NaN in one adapter's first factor, or in a row of
    another's second, reach its own tokens alone; without an adapter y is the
    residual."""
    n = 7
    g = torch.Generator().manual_seed(T)
    for ids in (torch.arange(T) % (n + 1) - 1, torch.randint(-1, n, (T,), generator=g), torch.arange(T) * n // T):
        c = Case(T, K, rank, rows, n, kind, ids=ids.tolist())
        want = c.run()
        for y, r in zip(want, c.resid):
            assert torch.equal(y[ids < 0], r[ids < 0])
        for bad in (float("inf"), float("-inf"), float("nan")):
            a, b = [t.clone() for t in c.a], [t.clone() for t in c.b]
            for m in range(len(rows)):
                c.a[m][2, rank - 1, K - 5] = bad
                c.b[m][4, rows[m] // 2, 3] = bad
                c.b[m][5, :, 0] = bad
            got = c.run()
            c.a, c.b = a, b
            for y, w, N in zip(got, want, rows):
                own, one = (ids == 2) | (ids == 5), ids == 4
                assert not torch.isfinite(y[own]).any()
                assert not torch.isfinite(y[one][:, N // 2]).any()
                y[one, N // 2] = w[one, N // 2]
                assert torch.equal(y[~own], w[~own]), bad


def _loose(c):
    """exact() with what is documented of small elements beside fp16 adapters,
    2^-43 of the token's largest, instead of an absolute bound."""
    step, extra = 2.0 ** -24, 8 if c.kind == "f16" else 0
    for a, b in zip(c.a, c.b):
        T, N = len(c.x), b.shape[1]
        y, tol = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
        for ad in range(len(a)):
            on = (c.ids == ad).nonzero()[:, 0]
            if not len(on):
                continue
            x, A, B = c.x[on].double(), a[ad].double(), b[ad].double()
            s = 1.0 if c.scale is None else float(c.scale[ad])
            v, mag = x @ A.t(), x.abs() @ A.abs().t()
            dv = (3 * c.K + 24 + extra) * step * mag
            if extra:
                dv += 2.0 ** -43 * x.abs().amax(1, keepdim=True) * A.abs().sum(1)
            d, dm = s * (v @ B.t()), abs(s) * (v.abs() @ B.abs().t())
            y[on] = d
            if extra: # the second factor's operand has the same two terms
                tol[on] = 2.0 ** -43 * abs(s) * v.abs().amax(1, keepdim=True) * B.abs().sum(1)
            tol[on] += abs(s) * (dv @ B.abs().t()) + (3 * c.rank + 8 + extra) * step * dm + 2 * step * d.abs()
        yield y, tol


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,K", [(1, 4096), (18, 256), (150, 1056), (300, 640)])
def test_inputs_of_any_size(T, K, kind):
    """From 1e-30 to 1e30, whole tokens of a size or sizes that rise and fall
    along a token; an adapter's result is as good relative to its input."""
    for factor in (1e-30, 1e-20, 1e-12, 1e-7, 1e-5, 1.0, 1e8, 1e20, 1e30):
        c = Case(T, K, 16, [64], 3, kind, ids=[i % 3 for i in range(T)], resid=False)
        c.x = c.x / c.x.abs().amax(1, keepdim=True) * factor
        for got, (y, tol) in zip(c.run(), _loose(c)):
            assert ((got.double() - y).abs() <= tol).all(), (kind, factor)
            # additions' errors have no common sign, and two fp16 terms are off by 2^-22
            assert float((got.double() - y).norm() / y.norm()) <= 2.0 ** -22 * (3 * K + 64) ** 0.5, (kind, factor)
    up = 10.0 ** torch.linspace(-30, 10, K)
    for shape in (up, up.flip(0), torch.where(torch.arange(K) % 7 == 3, 1e6, 1e-6), torch.where(torch.arange(K) >= K - 3, 1e9, 0.0)):
        c = Case(T, K, 16, [64], 3, kind, ids=[i % 3 for i in range(T)], resid=False)
        c.x = c.x / c.x.abs().amax(1, keepdim=True) * shape
        for got, (y, tol) in zip(c.run(), _loose(c)):
            assert ((got.double() - y).abs() <= tol).all(), kind


def test_a_token_does_not_see_its_neighbours_sizes():
    """fp16 operands are scaled by a power of two of the token's own."""
    for T in (20, 150, 300):
        c = Case(T, 512, 16, [64], 4, "f16", ids=[i % 4 for i in range(T)])
        want = c.run()[0]
        for t in range(0, T, 3):
            c.x[t] *= 1e12 if t % 2 else 1e-12
        got = c.run()[0]
        rest = [t for t in range(T) if t % 3]
        assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T", [1, 18, 300])
def test_small_elements_beside_a_large_one(T, kind):
    """The adapter does not look at the large one, and its result is the small
    ones' down to 2^-43 of the large one."""
    for large in (1.0, 1e15):
        for small in (2.0 ** -10, 2.0 ** -20, 2.0 ** -26, 2.0 ** -32, 2.0 ** -38):
            c = Case(T, 512, 16, [64], 3, kind, ids=[i % 3 for i in range(T)], resid=False)
            c.x = c.x / c.x.abs().amax(1, keepdim=True) * small * large
            for at in (0, 300, 511):
                c.x[:, at] = large
                for a in c.a:
                    a[:, :, at] = 0
            for got, (y, tol) in zip(c.run(), _loose(c)):
                assert ((got.double() - y).abs() <= tol).all(), (kind, large, small)
