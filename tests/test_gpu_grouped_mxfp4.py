"""Grouped products of bf16 rows with MXFP4 matrices, against a 64-bit form.

Tolerances. An activation enters as two terms that are within 2^-22 of its block's largest magnitude (2^-21 where that reaches
2^127), so a product sum is off by at most 2^-21 sum_k amax_k |b_k|; its fp32 sum of 2 K products by (2 K + 2) 2^-23 of the sum of
their magnitudes. The weights are exact. bf16 results round once more, 2^-8 of their magnitude at most; SiLU's slope is at most
1.1 and its __expf form within 2^-20 of it. Results scaled by a weight: one more fp32 rounding."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import mxfp4 as mx

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPI = {"store": L.LSK_EPI_STORE, "swiglu": L.LSK_EPI_SWIGLU, "scale": L.LSK_EPI_SCALE_F32}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    def __init__(self, sizes, N, K, epi="store", gather_k=0, seed=0, before=0, behind=0, gap=0):
        r = np.random.default_rng(seed * 7919 + sum(sizes) * 31 + N + K)
        E = len(sizes)
        bounds = before + np.concatenate(([0], np.cumsum(sizes)))
        self.E, self.N, self.K, self.epi, self.gather_k = E, N, K, epi, gather_k
        self.M = M = int(bounds[-1]) + behind
        self.at = bounds.tolist()
        self.bounds = _dev(bounds.astype(np.int32))
        rows = -(-M // gather_k) if gather_k else M
        a = r.standard_normal((max(rows, 1), K)) * np.exp2(r.integers(-6, 6, (max(rows, 1), 1)))
        self.A = _dev(a.astype(np.float32)).to(BF16)
        self.table = _dev(r.permutation(M).astype(np.int32))
        self.weight = _dev(r.random(M).astype(np.float32))
        self.codes, self.scales, self.values = [], [], []
        for _ in range(2 if epi == "swiglu" else 1):
            c, s = mx.encode(r.standard_normal((E * N, K)) * K ** -0.5)
            self.values.append(_dev(mx.decode(c, s, K).reshape(E, N, K)))
            self.codes.append(self._apart(_dev(c).reshape(E, N, -1), gap * 32))
            self.scales.append(self._apart(_dev(s).reshape(E, N, -1), gap * 16))
        self.out = torch.full((M + 1, N), 77.0, dtype=torch.float32 if epi == "scale" else BF16, device="cuda")

    @staticmethod
    def _apart(t, gap):
        if not gap:
            return t
        n = t[0].numel()
        wide = torch.full((t.shape[0], n + gap), 255, dtype=torch.uint8, device="cuda")
        wide[:, :n] = t.flatten(1)
        return wide[:, :n].unflatten(1, t.shape[1:])

    def run(self, stream=None):
        two = self.epi == "swiglu"
        L.lsk_gemm_grouped_bf16_mxfp4(
            EPI[self.epi], self.A, self.codes[0], self.scales[0], self.bounds, self.E, self.out, self.M, self.N, self.K,
            B2_codes=self.codes[1] if two else None, B2_scales=self.scales[1] if two else None, row_table=self.table,
            row_weight=self.weight if self.epi == "scale" else None, gather_k=self.gather_k, stream=stream)
        return self

    def exact(self):
        table = self.table.long()
        rows = self.A.double()
        rows = rows[table // self.gather_k] if self.gather_k else rows[:self.M]
        pad = torch.nn.functional.pad(rows.abs(), (0, -self.K % 32)).unflatten(1, (-1, 32)).amax(-1)
        amax = pad.repeat_interleave(32, 1)[:, :self.K]
        want = torch.full((self.M, self.N), float("nan"), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        for e in range(self.E):
            i, j = self.at[e], self.at[e + 1]
            if i == j:
                continue
            z, t = [], []
            for v in self.values:
                b = v[e]
                z.append(rows[i:j] @ b.T)
                t.append(2.0 ** -21 * (amax[i:j] @ b.abs().T) + (2 * self.K + 2) * 2.0 ** -23 * (rows[i:j].abs() @ b.abs().T))
            if self.epi == "swiglu":
                a = z[0] * torch.sigmoid(z[0])
                want[i:j] = a * z[1]
                tol[i:j] = 1.1 * t[0] * z[1].abs() + t[1] * (a.abs() + 1.1 * t[0]) + 2.0 ** -20 * want[i:j].abs()
            elif self.epi == "scale":
                w = self.weight.double()[table[i:j]][:, None]
                want[i:j], tol[i:j] = w * z[0], w * t[0] + 2.0 ** -24 * (w * z[0]).abs()
            else:
                want[i:j], tol[i:j] = z[0], t[0]
        if self.epi == "scale":
            w2, t2 = torch.full_like(want, float("nan")), torch.zeros_like(tol)
            w2[table], t2[table] = want, tol
            want, tol = w2, t2
        return want, tol

    def check(self):
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        want, tol = self.exact()
        got = self.out.double()
        left = torch.isnan(want)
        assert bool((got[:-1][left] == 77.0).all()) and bool((got[-1] == 77.0).all()), "wrote rows of no group"
        if self.out.dtype == BF16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38
        bad = ~left & ~((got[:-1] - want).abs() <= tol)
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: "
                                     f"{got[:-1][bad][0]} for {want[bad][0]}")


SIZES = [[1], [3, 0, 5], [16, 17, 1, 0, 0, 31], [0, 0, 33], [112, 113, 7], [300, 1, 0, 224, 225, 15], [1] * 200, [2, 700, 40], [64, 64, 64, 64]]
SHAPES = [(8, 8), (128, 128), (130, 136), (65, 520), (200, 1000), (768, 2048), (513, 768)]


@pytest.mark.parametrize("epi", list(EPI))
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_results_are_the_formulas(sizes, N, K, epi):
    sizes = sizes[:max(3, int(6e6 / (N * K)))]      # the oracle's time
    Case(sizes, N, K, epi).run().check()


@pytest.mark.parametrize("epi", list(EPI))
@pytest.mark.parametrize("k", [1, 3, 8])
@pytest.mark.parametrize("sizes", [[5, 0, 11], [60, 200, 3, 1]])
def test_rows_gathered_by_the_table(sizes, k, epi):
    Case(sizes, 136, 264, epi, gather_k=k).run().check()


@pytest.mark.parametrize("epi", list(EPI))
@pytest.mark.parametrize("sizes", [[0, 0], [4, 9], [250, 3]])
def test_rows_of_no_group_are_left_as_they_were(sizes, epi):
    Case(sizes, 72, 128, epi, before=5, behind=37, gap=3).run().check()


def test_bounds_are_cut_to_the_rows():
    c = Case([5, 7, 30], 72, 128, "store")
    c.bounds[0], c.bounds[3] = -100, 10 ** 6
    c.run().check()
    c = Case([5, 7, 30], 72, 128, "scale")
    c.table[3], c.table[9] = -1, 10 ** 6                       # no row of C
    was = c.out.clone()
    c.run()
    torch.cuda.synchronize()
    assert int((c.out == was).all(1).sum()) == 3 and L.lsk_device_error() == 0


@pytest.mark.parametrize("epi", ["store", "swiglu"])
@pytest.mark.parametrize("sizes", [[9, 20], [150, 200]])
def test_not_finite_values_stay_with_their_rows(sizes, epi):
    c = Case(sizes, 136, 200, epi).run()
    before = c.out.clone()
    c.A[4, 17], c.A[sizes[0] + 3, 5] = float("nan"), float("inf")
    c.run()
    torch.cuda.synchronize()
    own = torch.zeros(c.M + 1, dtype=torch.bool, device="cuda")
    own[4] = own[sizes[0] + 3] = True
    assert torch.equal(c.out[~own], before[~own]) and bool(torch.isnan(c.out[own]).all())
    c = Case(sizes, 136, 200, epi).run()
    c.scales[0][0, 3, 1] = 255                                  # a NaN block of one matrix's row
    c.run()
    torch.cuda.synchronize()
    hit = torch.isnan(c.out)
    assert bool(hit[:sizes[0], 3].all()) and int(hit.sum()) == sizes[0]


@pytest.mark.parametrize("sizes", [[3, 5, 0, 9], [40, 300, 0, 70]])
def test_captured_replayed_and_on_streams(sizes):
    cases = [Case(sizes, 264, 520, e, seed=i) for i, e in enumerate(EPI)]
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    first = [c.out.clone() for c in cases]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(stream=s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.out.fill_(77.0)
    torch.cuda.synchronize()
    for _ in range(10):
        for c, t, g in zip(cases, streams, graphs):
            with torch.cuda.stream(t):
                g.replay()
            c.run(stream=t)
    torch.cuda.synchronize()
    for c, f in zip(cases, first):
        assert torch.equal(c.out, f)
    # the same graph on other groups
    other = Case(list(reversed(sizes)), 264, 520, "store", seed=0)
    c = cases[0]
    c.A.copy_(other.A)
    c.bounds.copy_(other.bounds)
    c.at = other.at
    graphs[0].replay()
    c.check()


@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 256, 128), (64, 32, 4, 512, 256), (64, 128, 8, 2048, 768), (200, 16, 3, 264, 136)])
def test_a_layer_from_its_parts(T, E, k, H, F):
    """Routing, grouping, the experts' products and the sum: a layer with MXFP4 experts, and up to 64 tokens the same as lsk_moe_few."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    mats = {}
    for name, rows, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
        v = torch.randn((E * rows, K), generator=g, device="cuda") * K ** -0.5
        c = torch.empty((E, rows, L.lsk_mxfp4_code_pitch(K)), dtype=torch.uint8, device="cuda")
        s = torch.empty((E, rows, L.lsk_mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda")
        L.lsk_mxfp4_quantize(v, E * rows, K, c, s)
        back = torch.empty((E * rows, K), device="cuda")
        L.lsk_mxfp4_dequantize(c, s, E * rows, K, back)
        mats[name] = c, s, back.double().unflatten(0, (E, rows))
    sel = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    table = torch.empty(T * k, dtype=torch.int32, device="cuda")
    bounds = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    h = torch.empty((T * k, F), dtype=BF16, device="cuda")
    y = torch.empty((T * k, H), device="cuda")
    out, out32 = torch.empty_like(x), torch.empty((T, H), device="cuda")
    L.lsk_moe_route(logits, 1, T, E, k, sel, w)
    L.lsk_moe_group(sel, 1, T, E, k, table, bounds)
    L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SWIGLU, x, *mats["gate"][:2], bounds, E, h, T * k, F, H, B2_codes=mats["up"][0],
                                  B2_scales=mats["up"][1], row_table=table, gather_k=k)
    L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SCALE_F32, h, *mats["down"][:2], bounds, E, y, T * k, H, F, row_table=table, row_weight=w)
    L.lsk_moe_combine(x, y, T, k, H, out, out32)
    torch.cuda.synchronize()
    want, size = x.double(), x.double().abs()
    for t in range(T):
        for j in range(k):
            e = int(sel[t, j])
            a = mats["gate"][2][e] @ x[t].double()
            hid = a * torch.sigmoid(a) * (mats["up"][2][e] @ x[t].double())
            want[t] += float(w[t, j]) * (mats["down"][2][e] @ hid)
            size[t] += float(w[t, j]) * (mats["down"][2][e].abs() @ hid.abs())
    # the hidden activation's rounding to bf16, half a step of each value; the rest is far below it
    assert bool(((out32.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -12) * size).all())
    assert L.lsk_device_error() == 0
    if T <= 64:
        few = torch.empty((T, H), device="cuda")
        L.lsk_moe_few(x, logits, mats["gate"][0], mats["up"][0], mats["down"][0], T, E, k, H, F, out, gate_scales=mats["gate"][1],
                      up_scales=mats["up"][1], down_scales=mats["down"][1], out32=few)
        torch.cuda.synchronize()
        assert bool(((few - out32).abs().double() <= 2 * (2.0 ** -8 + 2.0 ** -12) * size).all())


@pytest.mark.parametrize("bounds", [[0, 25, 10, 30], [0, 250, 20, 300], [5, 200, 0, 300, 100, 280]])
def test_rows_that_bounds_out_of_order_give_to_two_groups_have_the_values_of_one(bounds):
    n, M = len(bounds) - 1, max(bounds)
    wants = []
    for e in range(n):
        c = Case([0] * e + [M] + [0] * (n - 1 - e), 130, 200)
        if e:
            c.codes, c.scales, c.values = first.codes, first.scales, first.values
        else:
            first = c
        want, tol = c.exact()
        wants.append((want, tol + 2.0 ** -8 * (want.abs() + tol)))
    first.bounds = _dev(np.array(bounds, np.int32))
    for _ in range(3):
        first.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    rows, got = torch.arange(M, device="cuda")[:, None], first.out[:M].double()
    right = torch.zeros_like(got, dtype=torch.bool)
    owned = torch.zeros_like(rows, dtype=torch.bool)
    for e, (want, tol) in enumerate(wants):
        mine = (rows >= bounds[e]) & (rows < bounds[e + 1])
        right |= mine & ((got - want).abs() <= tol)
        owned |= mine
    assert bool((right | ~owned).all()) and bool((got == 77.0)[~owned.expand_as(got)].all())


def test_no_rows_and_refusals():
    c = Case([4], 64, 64)
    c.M = 0
    c.run()
    for bad in ({"epi": L.LSK_EPI_RESID}, {"K": 60}, {"gather_k": -1}, {"N": 0}):
        a = {"epi": L.LSK_EPI_STORE, "N": 64, "K": 64, "gather_k": 0, **bad}
        with pytest.raises(L.LsError):
            L.lsk_gemm_grouped_bf16_mxfp4(a["epi"], c.A, c.codes[0], c.scales[0], c.bounds, 1, c.out, 4, a["N"], a["K"], row_table=c.table,
                                          gather_k=a["gather_k"])


@pytest.mark.parametrize("sizes", [[3, 2], [90, 7]])
def test_entries_of_the_table_that_are_no_row_count_as_zero(sizes):
    c = Case(sizes, 72, 128, "store", gather_k=4)
    c.table[1], c.table[4] = -1, 4 * c.A.shape[0]
    c.run()
    torch.cuda.synchronize()
    zero = (c.out[:-1] == 0).all(1)
    assert zero[1] and zero[4] and int(zero.sum()) == 2


@pytest.mark.parametrize("sizes", [[3, 0, 9], [130, 0, 250]])
@pytest.mark.parametrize("first", ["gate", "up"])
def test_gate_and_up_in_one_buffer_in_either_order(sizes, first):
    """Gate and up rows are read through one map where they can be: whichever lies first, and as one expert-major blob."""
    c = Case(sizes, 128, 256, "swiglu")
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    E, order = len(sizes), (0, 1) if first == "gate" else (1, 0)
    for kind in ("codes", "scales"):
        t = getattr(c, kind)
        blob = torch.stack([t[i] for i in order], 1).contiguous()          # [E, 2, N, pitch]
        setattr(c, kind, [blob[:, order.index(i)] for i in (0, 1)])
    c.out.fill_(77.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_calls_in_a_chain_overlap_without_harm():
    """Up, down and the next layer's up in a row, each started while the one before runs."""
    sizes, H, F = [40, 0, 9, 200, 64], 256, 384
    M = sum(sizes)
    up, down = Case(sizes, F, H, "swiglu", gather_k=1), Case(sizes, H, F, "scale")
    down.table, down.A = up.table, up.out[:M]
    want = []
    for times in (1, 25):
        for _ in range(times):
            up.run()
            if times == 1:
                torch.cuda.synchronize()
            down.run()
            if times == 1:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        want.append((up.out.clone(), down.out.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*want))


def test_captured_twice_and_replayed_in_turn():
    c = Case([5, 70, 0, 12], 264, 520, "scale")
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(stream=s)
            c.run(stream=s)
        graphs.append(g)
    for i in range(6):
        c.out.fill_(77.0)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
