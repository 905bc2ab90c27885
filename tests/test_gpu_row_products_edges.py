"""Products whose weights differ by rows, at the ends of what their arguments may be, and the precision of fp32 results."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import mxfp4 as mx
from test_gpu_grouped_mxfp4 import Case as Grouped
from test_gpu_grouped_mxfp4 import _dev
from test_gpu_lora import Case as Lora

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("epi", ["store", "swiglu", "scale"])
@pytest.mark.parametrize("M", [60, 300])          # single CTAs and pairs
@pytest.mark.parametrize("bounds", [[20, LOW, 0, 40, HIGH], [30, LOW, -7, HIGH, LOW], [LOW, 40, 41, HIGH, 45], [HIGH, 5, 50, LOW, LOW + 3],
                                    [16, LOW, LOW, LOW, LOW]], ids=lambda b: "_".join(map(str, b)))
def test_bounds_of_any_value_are_cut_to_the_rows(bounds, M, epi):
    """Row i is group g's where bounds[g] <= i < bounds[g + 1], and nothing else is written."""
    n = len(bounds) - 1
    wants = []
    for g in range(n):
        c = Grouped([0] * g + [M] + [0] * (n - 1 - g), 72, 128, epi)
        if g:
            c.codes, c.scales, c.values = first.codes, first.scales, first.values
        else:
            first = c
        want, tol = c.exact()
        wants.append((want, tol if epi == "scale" else tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38))
    first.bounds = _dev(np.array(bounds, np.int32))
    first.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    rows = torch.arange(M, device="cuda")
    place = first.table.long() if epi == "scale" else rows
    got = first.out[:M].double()
    assert bool((first.out[M] == 77.0).all())
    for g, (want, tol) in enumerate(wants):
        at = place[(rows >= bounds[g]) & (rows < bounds[g + 1])]
        assert bool(((got[at] - want[at]).abs() <= tol[at]).all()), g
    none = torch.ones(M, dtype=torch.bool, device="cuda")
    for g in range(n):
        none &= ~((rows >= bounds[g]) & (rows < bounds[g + 1]))
    assert bool((got[place[none]] == 77.0).all())


# exponent fields of blocks of 32: subnormal, next to either border of the split's quick form and of the range, ordinary; -1: zeros
FIELDS = [0, 127, -1, 1, 31, 0, 32, 33, 253, 254, 0, 0, 127, 12]


@pytest.mark.parametrize("epi", ["store", "scale"])
@pytest.mark.parametrize("sizes", [[9, 20], [150, 200]])
@pytest.mark.parametrize("fields", [FIELDS, [0] * 8, [0, -1, 127, 200] * 4, [31, 0] * 5], ids=lambda f: "_".join(map(str, f)))
def test_blocks_of_every_magnitude_count_alike(fields, sizes, epi):
    """Weights whose blocks undo the rows' magnitudes, so that a block's part of the result does not drown in another's."""
    N, K = 136, 32 * len(fields)
    c = Grouped(sizes, N, K, epi)
    r = np.random.default_rng(len(fields))
    f = np.array(fields)[np.stack([r.permutation(len(fields)) for _ in range(2)])]       # an order of blocks for each group
    c.codes, c.scales, c.values, bits = [], [], [], []
    for e in range(2):
        field = f[e].repeat(32)
        mant = np.where(r.random((sizes[e], K)) < 0.3, r.integers(0x78, 0x80, (sizes[e], K)), r.integers(1, 0x80, (sizes[e], K)))
        bits.append(np.where(field < 0, 0, r.integers(0, 2, (sizes[e], K)) << 15 | np.maximum(field, 0) << 7 | mant).astype(np.uint16))
        codes, scales = mx.encode(r.standard_normal((N, K)) * np.exp2(np.clip(127.0 - field, -120, 120)))
        c.values.append(_dev(mx.decode(codes, scales, K)))
        c.codes.append(_dev(codes))
        c.scales.append(_dev(scales))
    c.values, c.codes, c.scales = [torch.stack(c.values)], [torch.stack(c.codes)], [torch.stack(c.scales)]
    c.A = _dev(np.concatenate(bits).view(np.int16)).view(torch.bfloat16)
    c.run().check()


@pytest.mark.parametrize("M", [40, 640])
def test_gates_far_below_zero_keep_their_share(M):
    """SiLU(g) = g / (1 + e^-g) beyond the g where e^-g leaves the range of fp32 or of a fast division, beside up values that bring
    it back. e^g by __expf is within 2 + 1.173 |g| units in the last place, 2^-16 of it for these g, and within 2^-149 where it is
    subnormal; a product with g that is subnormal within 2^-150 more; the result's rounding 2^-8."""
    K, N = 64, 24
    one, other = np.zeros((N, K)), np.zeros((N, K))
    one[:, 0] = one[:, 1] = 1.0
    other[:, 32] = 1.0
    (gc, gs), (uc, us) = mx.encode(one), mx.encode(other)
    i = np.arange(M) * 640 // M
    A = torch.zeros((M, K))
    A[:, 0], A[:, 1], A[:, 32] = torch.from_numpy(-60.0 - i // 16), torch.from_numpy(-(i % 16) / 16.0), 2.0 ** 110     # gates -60 to -99.9
    out = torch.full((M + 1, N), 77.0, dtype=torch.bfloat16, device="cuda")
    b = _dev(np.array([0, M], np.int32))
    L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SWIGLU, A.to(torch.bfloat16).cuda(), _dev(gc)[None], _dev(gs)[None], b, 1, out, M, N, K,
                                  B2_codes=_dev(uc)[None], B2_scales=_dev(us)[None])
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0 and bool((out[M] == 77.0).all())
    g = (A[:, 0] + A[:, 1]).double().cuda()[:, None]
    want = g * torch.sigmoid(g) * 2.0 ** 110
    tol = 2.0 ** -16 * want.abs() + (g.abs() + 1) * 2.0 ** -149 * 2.0 ** 110
    assert bool(((out[:M].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


# The precision of fp32 results, by norm: a bound on each value as the other tests have it (K 2^-23 of the sum of magnitudes) would let
# a single long chain of tensor core sums pass, and h in two terms. A tensor core cuts its sums off: a product takes in 16 values of K
# and loses half of a last bit on average, 2^-25 of the sum so far, always towards zero. A chain of c stages of 64 values is 4 c products,
# so a result is off by at most 4 c 2^-25 of its norm. Fewer additions in registers than products follow, and the last
# roundings: 2^-23. (Two terms of h instead of three are off by up to 2^-18 of it.)
def _cut(products):
    return products * 2.0 ** -25 + 2.0 ** -23


def _error(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,K,r,n,stages", [(20, 256, 16, 4, 1), (64, 200, 40, 9, 1), (20, 13824, 32, 8, 16), (128, 13824, 256, 128, 16), (128, 13824, 8, 128, 16),
                                            (70, 40000, 16, 3, 16), (300, 256, 24, 5, 2), (300, 13824, 16, 3, 16), (4096, 13824, 64, 64, 16),
                                            (2100, 30000, 136, 40, 16), (16384, 13824, 16, 2, 16)])
def test_the_adapters_part_alone_has_its_24_bits(T, K, r, n, stages):
    """h from many slices of K and from few (many rows, many adapters, a long K): chains of 16 stages at most."""
    c = Lora(T, 136, K, r, n, "resid_only", seed=1)
    c.w.zero_()
    c.resid.zero_()
    c.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    want = torch.zeros((T, 136), dtype=torch.float64, device="cuda")
    for a in range(n):
        rows = torch.nonzero(c.ids == a).flatten()
        want[rows] = float(c.scale[a]) * (c.x[rows].double() @ c.down[a].double().T) @ c.up[a].double().T
    up = min(3 * -(-r // 16), 4 * 16)             # products of the adapter's own chain
    assert _error(c.out32[:T], want) <= _cut(4 * stages + up)


@pytest.mark.parametrize("epi", ["resid", "resid_only"])
@pytest.mark.parametrize("T,N,K", [(1, 520, 13824), (16, 136, 5120), (64, 1000, 13824), (128, 264, 5120), (128, 2560, 13824), (129, 264, 5120), (300, 520, 13824),
                                   (1024, 2056, 5120), (700, 136, 2048), (300, 1024, 1024)])
def test_the_shared_part_alone_is_summed_in_short_chains(T, N, K, epi):
    c = Lora(T, N, K, 16, 3, epi, ids=[-1] * T, seed=2)
    c.resid.zero_()
    if c.bias is not None:
        c.bias.zero_()
    c.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    stages = 4 if T <= 128 else 8 if K <= 2048 else 16
    assert _error(c.out32[:T], c.x.double() @ c.w.double().T) <= _cut(4 * stages)


@pytest.mark.parametrize("T,K,r,n", [(70, 40000, 16, 3), (1500, 30000, 136, 40)])
def test_long_slices_in_flight_captured_and_again_the_same_bits(T, K, r, n):
    """Calls whose h is summed in rounds: three of them on streams of their own, then two captured ones replayed in turn."""
    cases = [Lora(T, 200, K, r, n, "resid", seed=s) for s in range(3)]
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    first = [(c.out.clone(), c.out32.clone()) for c in cases]

    def same():
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        for c, (a, b) in zip(cases, first):
            assert torch.equal(c.out, a) and torch.equal(c.out32, b)
            c.out[:T].fill_(0)       # not the row behind the last
            c.out32[:T].fill_(0)

    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    same()
    graphs = []
    for c in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            c.run(stream=streams[0])
        graphs.append(g)
    cases[2].run()
    for _ in range(4):
        for g in graphs:
            g.replay()
    same()
