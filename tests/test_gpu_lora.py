"""The shared projection with low-rank adapters beside it, against a 64-bit form.

Tolerances. The fp32 sum of n products of bf16 values, in whatever order, is within n 2^-23 sum|products| of the exact one; the
two terms of h are within 2^-16 |h| (the three of a call with fp32 results within 2^-23), and h itself within K 2^-23 of its own sum of magnitudes. So a result before the epilogue
is within  (K + r + 4) 2^-23 S + 2^-16 S_h,  where S is the sum of all magnitudes |x w| and |s||x d||u|, and S_h that of the
adapter's part; far less in fact. A bf16 result is then rounded once: half a step, 2^-8 of its magnitude at most. GELU and SiLU
have slopes of at most 1.13 and 1.1; GELU's own form is within 2e-6 of the exact one, SiLU's by __expf within 2^-20 relative."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPI = {"store": L.LSK_EPI_STORE, "gelu": L.LSK_EPI_BIAS_GELU, "resid": L.LSK_EPI_BIAS_RESID, "swiglu": L.LSK_EPI_SWIGLU,
       "resid_only": L.LSK_EPI_RESID}


class Case:
    def __init__(self, T, N, K, r, n, epi="store", ids=None, seed=0, resid_f32=True, scaled=True, gap=0):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + T + N + K)

        def normal(*shape, scale=1.0, dtype=BF16):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

        two = 2 if epi == "swiglu" else 1
        self.T, self.N, self.K, self.r, self.n, self.epi, self.two = T, N, K, r, n, epi, two
        self.x = normal(T, K)
        self.w = normal(two * N, K, scale=K ** -0.5)
        self.down = normal(n, two * r * K + gap, scale=K ** -0.5)[:, :two * r * K].unflatten(1, (two * r, K))
        self.up = normal(n, N * r + gap, scale=r ** -0.5)[:, :N * r].unflatten(1, (N, r))
        self.up2 = normal(n, N * r + gap, scale=r ** -0.5)[:, :N * r].unflatten(1, (N, r)) if two == 2 else None
        self.scale = 0.25 + torch.rand(n, generator=g, device="cuda") if scaled else None
        self.bias = normal(N, scale=0.5) if epi in ("gelu", "resid") else None
        self.resid = normal(T, N, dtype=torch.float32 if resid_f32 else BF16) if epi.startswith("resid") else None
        ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32) if ids is None else ids
        self.ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda")
        self.out = torch.full((T + 1, N), 77.0, dtype=BF16, device="cuda")
        self.out32 = torch.full((T + 1, N), 77.0, device="cuda") if epi.startswith("resid") else None

    def run(self, stream=None):
        self.lora = L.lsk_lora_adapters(self.down, self.up, up2=self.up2, scale=self.scale)
        L.lsk_gemm_lora_bf16(EPI[self.epi], self.x, self.w, self.lora, self.ids, self.out, self.T, self.N, self.K, bias=self.bias,
                             resid=self.resid, b2_row_off=self.N if self.two == 2 else 0, C32=self.out32, stream=stream)
        return self

    def exact(self):
        """The result in 64 bits and the bound on what the kernel may be off by before the last rounding."""
        x, ids = self.x.double(), self.ids.long()
        N, r = self.N, self.r
        parts, tols = [], []
        for half in range(self.two):
            w = self.w[half * N:(half + 1) * N].double()
            z, S = x @ w.T, x.abs() @ w.abs().T
            Sh = torch.zeros_like(z)
            for a in range(self.n):
                rows = torch.nonzero(ids == a).flatten()
                if not len(rows):
                    continue
                s = 1.0 if self.scale is None else float(self.scale[a])
                d = self.down[a, half * r:(half + 1) * r].double()
                u = (self.up2 if half else self.up)[a].double()
                z[rows] += s * (x[rows] @ d.T) @ u.T
                Sh[rows] = abs(s) * (x[rows].abs() @ d.abs().T) @ u.abs().T
            parts.append(z)
            tols.append((self.K + r + 4) * 2.0 ** -23 * (S + Sh) + (2.0 ** -16 if self.out32 is None else 2.0 ** -23) * Sh)
        z, tol = parts[0], tols[0]
        if self.epi == "swiglu":
            g, u = parts
            a = g * torch.sigmoid(g)
            return a * u, 1.1 * tols[0] * u.abs() + tols[1] * (a.abs() + 1.1 * tols[0]) + 2.0 ** -20 * (a * u).abs()
        if self.bias is not None:
            z = z + self.bias.double()
        if self.epi == "gelu":
            return z * torch.special.ndtr(z), 1.13 * tol + 2e-6 * (1 + z.abs())
        if self.resid is not None:
            z = z + self.resid.double()
        return z, tol + 2.0 ** -22 * z.abs()

    def check(self):
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        want, tol = self.exact()
        got = self.out[:self.T].double()
        bad = ~((got - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38)
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: "
                                     f"{got[bad][0]} for {want[bad][0]}")
        assert bool((self.out[self.T:] == 77.0).all()), "wrote past the last row"
        if self.out32 is not None:
            assert bool(((self.out32[:self.T].double() - want).abs() <= tol).all())
            assert bool((self.out32[self.T:] == 77.0).all())


SHAPES = [(1, 128, 64, 8, 1), (1, 8, 8, 8, 3), (3, 200, 72, 16, 2), (16, 1096, 1000, 24, 8), (17, 256, 2048, 32, 5), (33, 640, 520, 40, 40),
          (64, 1000, 1024, 64, 64), (65, 136, 136, 72, 9), (100, 2048, 512, 128, 6), (128, 512, 640, 256, 3), (129, 512, 256, 16, 3),
          (256, 1024, 1000, 32, 300), (300, 1048, 192, 64, 17), (513, 2000, 328, 120, 4), (700, 256, 64, 256, 2), (1025, 160, 1024, 8, 1)]


@pytest.mark.parametrize("epi", list(EPI))
@pytest.mark.parametrize("T,N,K,r,n", SHAPES)
def test_results_are_the_formulas(T, N, K, r, n, epi):
    Case(T, N, K, r, n, epi).run().check()


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("epi", ["store", "swiglu", "resid"])
def test_rows_without_an_adapter_have_the_shared_product(T, epi):
    ids = [[-1, 5, 6, -7, 2 ** 31 - 1][i % 5] for i in range(T)]      # five adapters: none of these is one
    c = Case(T, 264, 320, 16, 5, epi, ids=ids)
    c.run().check()
    c.ids = torch.full_like(c.ids, -1)
    want = Case(T, 264, 320, 16, 5, epi, ids=[-1] * T)
    want.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want.out)


@pytest.mark.parametrize("T,reqs", [(64, 1), (64, 64), (300, 3), (1024, 7), (1024, 1024)])
def test_rows_in_runs_and_one_by_one(T, reqs):
    ids = (torch.arange(T) * reqs // T) % 96
    Case(T, 384, 256, 16, 96, "store", ids=ids).run().check()


@pytest.mark.parametrize("T", [20, 200])
def test_adapters_apart_unscaled_and_bf16_residual(T):
    Case(T, 256, 256, 16, 4, "resid", resid_f32=False, scaled=False, gap=24).run().check()


@pytest.mark.parametrize("T", [1, 31, 128, 300])
@pytest.mark.parametrize("epi", ["store", "swiglu"])
@pytest.mark.parametrize("where", ["up", "up2", "down", "scale"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_adapter_that_is_not_finite_stays_with_its_own_rows(T, epi, where, value):
    if where == "up2" and epi == "store":
        pytest.skip("one projection")
    c = Case(T, 200, 128, 16, 4, epi, ids=[(i // 3) % 5 - 1 for i in range(T)])
    want = Case(T, 200, 128, 16, 4, epi, ids=[-1 if (i // 3) % 5 == 3 else (i // 3) % 5 - 1 for i in range(T)])
    want.run()
    if where == "scale":
        c.scale[2] = value
    else:
        getattr(c, where)[2, 3, 5] = value
    c.run()
    torch.cuda.synchronize()
    own = c.ids == 2
    assert torch.equal(c.out[:T][~own], want.out[:T][~own])
    assert not bool(own.any()) or bool(~torch.isfinite(c.out[:T][own]).all())


@pytest.mark.parametrize("T", [9, 300])
def test_a_row_that_is_not_finite_stays_alone(T):
    c = Case(T, 200, 128, 16, 4).run()
    before = c.out.clone()
    c.x[7, 5] = float("inf")
    c.run()
    torch.cuda.synchronize()
    keep = torch.arange(T + 1, device="cuda") != 7
    assert torch.equal(c.out[keep], before[keep]) and not bool(torch.isfinite(c.out[7]).any())


def test_weights_in_a_larger_matrix():
    """b_rows above N: the rows after the projection's are another's."""
    c = Case(50, 136, 256, 16, 3)
    big = torch.full((500, 256), float("nan"), dtype=BF16, device="cuda")
    big[:136] = c.w
    c.w = big
    c.run()
    c.w = big[:136]
    c.check()


@pytest.mark.parametrize("T", [5, 64, 300])
def test_captured_and_replayed_on_other_inputs(T):
    """Two graphs of the same call, replayed in turn on changed inputs and ids."""
    c = Case(T, 512, 512, 16, 6, "gelu")
    c.run()
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(stream=s)
        graphs.append(g)
    for i in range(4):
        other = Case(T, 512, 512, 16, 6, "gelu", seed=i + 1)
        c.x.copy_(other.x)
        c.ids.copy_(other.ids)
        graphs[i % 2].replay()
        c.check()


@pytest.mark.parametrize("T", [16, 300])
def test_calls_in_flight_on_streams_and_again_the_same_bits(T):
    cases = [Case(T, 1024, 512, 16, 8, e, seed=i) for i, e in enumerate(("store", "swiglu", "resid"))]
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    first = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, f in zip(cases, first):
        assert torch.equal(c.out, f)
        c.check()


def test_no_rows():
    c = Case(4, 64, 64, 8, 2)
    assert L.lsk_gemm_lora_bf16(L.LSK_EPI_STORE, c.x, c.w, L.lsk_lora_adapters(c.down, c.up), c.ids, c.out, 0, 64, 64) == L.LS_OK


@pytest.mark.parametrize("T,K,r", [(3, 6400, 16), (5, 8000, 16), (2, 11000, 16), (20, 13824, 32), (70, 8192, 64), (100, 4104, 256), (150, 13824, 16), (260, 9000, 128)])
def test_long_rows_shared_by_clusters_of_every_size(T, K, r):
    Case(T, 256, K, r, 3, "swiglu", seed=3).run().check()


@pytest.mark.parametrize("T", [30, 200])
def test_many_adapters(T):
    """More than the numbers that the notes on adapters tell apart; two in use share one, and one of them is not finite."""
    n, ids = 5000, [[7, 7 + 4096, 4999, 0, 2500][i % 5] for i in range(T)]
    c = Case(T, 64, 64, 8, n, "store", ids=ids).run()
    c.check()
    before = c.out.clone()
    c.up[7 + 4096, 3, 2] = float("inf")
    c.run()
    torch.cuda.synchronize()
    own = torch.zeros(T + 1, dtype=torch.bool, device="cuda")
    own[:T] = c.ids == 7 + 4096
    assert torch.equal(c.out[~own], before[~own]) and not bool(torch.isfinite(c.out[own]).all(1).any())


@pytest.mark.parametrize("T,K,r,n,used", [(90, 4096, 8, 77, 11), (96, 4096, 16, 96, 11), (64, 2048, 32, 64, 11), (300, 4096, 32, 3, 2)])
def test_sums_of_a_cluster_are_whole_before_they_are_added(T, K, r, n, used):
    """Many calls one behind the other, each with other rows of x: no row may have sums of the call before, or none."""
    cases = [Case(T, 200, K, r, n, ids=[(7 * i) % used + (n - used) for i in range(T)], seed=s) for s in range(4)]
    wants = [c.exact() for c in cases]
    for _ in range(25):
        for c in cases:
            c.run()
        torch.cuda.synchronize()
        for c, (want, tol) in zip(cases, wants):
            assert bool(((c.out[:T].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


@pytest.mark.parametrize("epi", ["store", "swiglu", "resid"])
@pytest.mark.parametrize("T,K,r,n,used", [(128, 640, 16, 128, 128), (90, 4096, 8, 77, 77), (64, 2048, 32, 64, 11), (16, 1032, 24, 9, 3), (9, 512, 64, 9, 5),
                                          (48, 1024, 40, 40, 7), (128, 8192, 32, 8, 8)])
def test_gangs_of_few_rows_adapters(T, K, r, n, used, epi):
    """Numbers of adapters that leave the last gang of a slot short, in use by rows apart."""
    ids = [(7 * i) % used + (n - used) for i in range(T)]
    Case(T, 200, K, r, n, epi, ids=ids, seed=5).run().check()


@pytest.mark.parametrize("epi", ["resid", "resid_only"])
@pytest.mark.parametrize("T,N,K,r,n", [(700, 8008, 1096, 72, 9), (520, 7000, 2312, 256, 3), (1100, 4096, 2048, 8, 1100), (257, 200, 8, 16, 1)])
def test_chains_of_fp32_results_over_several_tiles(T, N, K, r, n, epi):
    """More tiles than pairs of SMs, chains cut short by the end of K and of the adapters, every id none's in some rows."""
    Case(T, N, K, r, n, epi, seed=7).run().check()
    Case(T, N, K, r, n, epi, ids=[-1] * T, seed=7).run().check()


@pytest.mark.parametrize("T", [40, 300])
def test_the_residual_stream_in_place(T):
    """C32 over the residual that it takes: every element is read before it is written."""
    c = Case(T, 512, 256, 16, 4, "resid")
    c.run()
    torch.cuda.synchronize()
    first = c.out.clone(), c.out32.clone()
    both = torch.empty((T + 1, 512), device="cuda")
    both[:T], both[T] = c.resid, 77.0
    c.resid, c.out32 = both[:T], both
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first[0]) and torch.equal(c.out32, first[1])


def test_behind_and_before_other_products_of_the_library():
    """The product starts while the kernel before it runs: calls in a chain, each on what the one before wrote."""
    T, H, F = 48, 512, 1024
    up, down = Case(T, F, H, 16, 4, "gelu"), Case(T, H, F, 16, 4, "resid", resid_f32=False)
    down.ids, down.x, down.resid = up.ids, up.out[:T], up.x
    want = []
    for overlapped in (False, True):
        up.out.fill_(0)
        for _ in range(1 if not overlapped else 30):
            up.run()
            if not overlapped:
                torch.cuda.synchronize()
            down.run()
            if not overlapped:
                torch.cuda.synchronize()
            L.lsk_gemm_bf16(L.LSK_EPI_BIAS_GELU, up.x, up.w, up.out, T, F, H, bias=up.bias)   # over the rows that were just read
            if not overlapped:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        want.append((down.out.clone(), down.out32.clone(), up.out.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*want))
