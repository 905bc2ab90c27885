"""The few-token MoE layer against the 64-bit oracle, with bf16 and MXFP4 experts."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import forward as F64
from oracle import mxfp4 as mx

from gpu_util import bf16_dev, rand_bf16, to_f64

pytestmark = pytest.mark.gpu


class Layer:
    """Random experts on the device (optionally inside wider blobs) and their values."""

    def __init__(self, E, H, F, mx4, seed, gap=0):
        self.E, self.H, self.F, self.mx4 = E, H, F, mx4
        self.values, self.args = {}, {}
        for i, (name, rows, K) in enumerate((("gate", F, H), ("up", F, H), ("down", H, F))):
            if mx4:
                v = np.random.default_rng(seed + i).standard_normal((E * rows, K)) * K ** -0.5
                c, s = mx.encode(v)
                self.values[name] = mx.decode(c, s, K).reshape(E, rows, K)
                self.args[name] = self._place(torch.from_numpy(c).reshape(E, rows, -1), gap)
                self.args[name + "_scales"] = self._place(torch.from_numpy(s).reshape(E, rows, -1), gap)
            else:
                b, v = rand_bf16((E, rows, K), seed + i, K ** -0.5)
                self.values[name] = v
                self.args[name] = self._place(torch.from_numpy(b.view(np.int16)).view(torch.bfloat16), gap)

    @staticmethod
    def _place(t, gap):
        """[E, rows, cols] with `gap` extra rows' bytes (a multiple of 64) between experts."""
        E, rows, cols = t.shape
        buf = torch.zeros((E, rows * cols + gap * 64), dtype=t.dtype)
        buf[:, :rows * cols] = t.reshape(E, -1)
        return buf.cuda()[:, :rows * cols].unflatten(1, (rows, cols))

    def run(self, x, logits, k, out=None, **kw):
        T = x.shape[0]
        out = torch.full((T + 1, self.H), 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        a = self.args
        scales = {n: a[n] for n in ("gate_scales", "up_scales", "down_scales") if n in a}
        L.lsk_moe_few(x, logits, a["gate"], a["up"], a["down"], T, self.E, k, self.H, self.F, out, **scales, **kw)
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        return out

    def reference(self, x, logits, k, r=None):
        """(out, tolerance before the rounding of the output): each step's roundings carried through."""
        sel, w = F64.route_topk(logits, k)
        y = (x if r is None else r).copy()
        tol = 2.0 ** -22 * np.abs(y)
        eps_sum = lambda K: (K / 32 + 8) * 2.0 ** -22  # noqa: E731
        for t in range(x.shape[0]):
            for j in range(k):
                G, U, D = (self.values[n][sel[t, j]] for n in ("gate", "up", "down"))
                g, u = G @ x[t], U @ x[t]
                s = F64.silu(g)
                h = s * u
                # sums; with 4-bit experts x is held to 2^-22 of its largest value
                ax = np.abs(x[t]) * eps_sum(self.H) + (2.0 ** -22 * np.abs(x[t]).max() if self.mx4 else 0.0)
                dg, du = np.abs(G) @ ax, np.abs(U) @ ax
                hmax = np.abs(np.pad(h, (0, -self.F % 32))).reshape(-1, 32).max(1).repeat(32)[:self.F]
                dh = 1.1 * np.abs(u) * dg + np.abs(s) * du + 2.0 ** -18 * np.abs(h)
                dh += 2.0 ** -11 * np.abs(h) + 2.0 ** -22 * hmax if self.mx4 else 2.0 ** -9 * np.abs(h)
                y[t] += w[t, j] * (D @ h)
                tol[t] += w[t, j] * (np.abs(D) @ (dh + eps_sum(self.F) * np.abs(h))) + 2.0 ** -20 * np.abs(w[t, j] * (D @ h))
        return y, tol


def _check(out, ref, tol):
    got = to_f64(out[:ref.shape[0]])
    tol = tol + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)
    if out.shape[0] > ref.shape[0]:
        assert bool((out[ref.shape[0]] == 77.0).all()), "wrote past the last token"


CASES = [(1, 1, 1, 8, 8), (1, 8, 2, 264, 40), (1, 128, 8, 512, 264), (2, 3, 3, 520, 96), (7, 60, 4, 1048, 520),
         (16, 16, 8, 256, 768), (17, 8, 2, 520, 136), (33, 256, 8, 136, 72), (64, 128, 8, 264, 128), (64, 4, 4, 128, 64)]


@pytest.mark.parametrize("T,E,k,H,F", CASES)
@pytest.mark.parametrize("mx4", [False, True])
def test_layer_vs_oracle(T, E, k, H, F, mx4):
    layer = Layer(E, H, F, mx4, T + E)
    xb, x = rand_bf16((T, H), 50)
    lg = np.random.default_rng(51).standard_normal((T, E)).astype(np.float32)
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k)
    _check(out, *layer.reference(x, lg, k))


@pytest.mark.parametrize("T,E,k,H,F", [(7, 60, 4, 1048, 520), (40, 64, 8, 776, 328), (64, 64, 2, 1160, 584)])
@pytest.mark.parametrize("mx4", [False, True])
def test_many_units_of_an_odd_number_of_stages(T, E, k, H, F, mx4):
    """A stage of the ring changes between even and odd places of a unit: its waits must not take an older round for theirs."""
    layer = Layer(E, H, F, mx4, 91)
    xb, x = rand_bf16((T, H), 92)
    lg = np.random.default_rng(93).standard_normal((T, E)).astype(np.float32)
    x_dev, lg_dev = bf16_dev(xb), torch.from_numpy(lg).cuda()
    out = layer.run(x_dev, lg_dev, k)
    _check(out, *layer.reference(x, lg, k))
    for _ in range(20):
        assert torch.equal(layer.run(x_dev, lg_dev, k), out)


@pytest.mark.parametrize("mx4", [False, True])
def test_blobs_residual_stream_and_fp32_output(mx4):
    T, E, k, H, F = 5, 6, 2, 264, 96
    layer = Layer(E, H, F, mx4, 3, gap=3)
    xb, x = rand_bf16((T, H), 52)
    r = np.random.default_rng(53).standard_normal((T, H)).astype(np.float32)
    lg = np.random.default_rng(54).standard_normal((T, E)).astype(np.float32)
    out32 = torch.empty((T, H), dtype=torch.float32, device="cuda")
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k, resid=torch.from_numpy(r).cuda(), out32=out32)
    ref, tol = layer.reference(x, lg, k, r.astype(np.float64))
    assert np.all(np.abs(to_f64(out32) - ref) <= tol)
    assert torch.equal(out[:T], out32.to(torch.bfloat16))


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [15, 16, 17, 64])
def test_every_token_on_the_same_experts(mx4, T):
    E, k, H, F = 9, 3, 256, 64
    layer = Layer(E, H, F, mx4, 5)
    xb, x = rand_bf16((T, H), 55)
    lg = np.tile(np.arange(E, dtype=np.float32) * 0.25, (T, 1))
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k)
    _check(out, *layer.reference(x, lg, k))


@pytest.mark.parametrize("mx4", [False, True])
def test_unrouted_experts_are_not_read_into_the_result(mx4):
    T, E, k, H, F = 4, 20, 2, 128, 64
    layer = Layer(E, H, F, mx4, 7)
    xb, x = rand_bf16((T, H), 56)
    lg = np.random.default_rng(57).standard_normal((T, E)).astype(np.float32)
    ref, tol = layer.reference(x, lg, k)
    used = set(F64.route_topk(lg, k)[0].reshape(-1).tolist())
    for e in set(range(E)) - used:
        for n, t in layer.args.items():
            if n.endswith("scales") or not mx4:
                t[e] = 255 if mx4 else float("nan")
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k)
    _check(out, ref, tol)


@pytest.mark.parametrize("mx4", [False, True])
def test_routing_of_ties_masks_and_nan(mx4):
    T, E, k, H, F = 6, 40, 4, 128, 64
    layer = Layer(E, H, F, mx4, 9)
    xb, x = rand_bf16((T, H), 58)
    lg = np.random.default_rng(59).standard_normal((T, E)).astype(np.float32)
    lg[0] = 1.0                                    # all equal: experts 0 to 3
    lg[1, ::2] = 0.0
    lg[1, 1::2] = -0.0                             # zeros of both signs are equal
    lg[2] = -np.inf                                # nothing left: the residual alone
    lg[3, 3:] = -np.inf                            # three experts and one of weight 0
    lg[4, 7] = np.nan                              # not among the largest
    lg[5, 4:] = np.nan                             # four numbers, all chosen
    clean = np.where(np.isnan(lg), -np.inf, lg)
    clean[2] = 0.0
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k)
    ref, tol = layer.reference(x, clean, k)
    ref[2], tol[2] = x[2], 0.0
    _check(out, ref, tol)
    lg[4] = np.nan
    out = layer.run(bf16_dev(xb), torch.from_numpy(lg).cuda(), k)
    assert bool(torch.isnan(out[4]).all()) and bool(torch.isfinite(out[[0, 1, 2, 3, 5]]).all())


@pytest.mark.parametrize("mx4", [False, True])
def test_tokens_of_very_different_size_and_non_finite_ones_stay_apart(mx4):
    T, E, k, H, F = 5, 8, 2, 256, 96
    layer = Layer(E, H, F, mx4, 11)
    xb, x = rand_bf16((T, H), 60)
    t = bf16_dev(xb)
    scale = torch.tensor([2.0 ** -40, 1.0, 2.0 ** 20, 1.0, 1.0], device="cuda").bfloat16()
    t = t * scale[:, None]
    x = x * scale.double().cpu().numpy()[:, None]
    t[3, 5] = float("nan")
    t[4, 7] = float("inf")
    lg = np.random.default_rng(61).standard_normal((T, E)).astype(np.float32)
    out = layer.run(t, torch.from_numpy(lg).cuda(), k)
    ref, tol = layer.reference(x, lg, k)
    _check(out[:3], ref[:3], tol[:3])
    assert bool(torch.isnan(out[3]).all()) and not bool(torch.isfinite(out[4]).all())


@pytest.mark.parametrize("mx4", [False, True])
def test_same_bits_every_time_on_any_stream_and_in_a_graph(mx4):
    T, E, k, H, F = 12, 32, 4, 512, 256
    layer = Layer(E, H, F, mx4, 13)
    xb, _ = rand_bf16((T, H), 62)
    x = bf16_dev(xb)
    lg = torch.from_numpy(np.random.default_rng(63).standard_normal((T, E)).astype(np.float32)).cuda()
    first = layer.run(x, lg, k)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(layer.run(x, lg, k, stream=streams[i % 2]), first)
    out = torch.zeros_like(first)
    a = layer.args
    scales = {n: a[n] for n in ("gate_scales", "up_scales", "down_scales") if n in a}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lsk_moe_few(x, lg, a["gate"], a["up"], a["down"], T, E, k, H, F, out, **scales)
    for _ in range(2):
        out[:T] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:T], first[:T])


def test_layer_agrees_with_the_grouped_path():
    """The same layer through route, group, gather, the grouped GEMMs and combine."""
    T, E, k, H, F = 9, 16, 4, 256, 128
    layer = Layer(E, H, F, False, 15)
    xb, x = rand_bf16((T, H), 64)
    lg = torch.from_numpy(np.random.default_rng(65).standard_normal((T, E)).astype(np.float32)).cuda()
    xd = bf16_dev(xb)
    sel = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), dtype=torch.float32, device="cuda")
    table = torch.empty(T * k, dtype=torch.int32, device="cuda")
    bounds = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    L.lsk_moe_route(lg, 1, T, E, k, sel, w)
    L.lsk_moe_group(sel, 1, T, E, k, table, bounds)
    xs = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    L.lsk_moe_gather(xd, table, T * k, k, H, xs)
    both = torch.cat((layer.args["gate"].reshape(E * F, H), layer.args["up"].reshape(E * F, H))).contiguous()
    h = torch.empty((T * k, F), dtype=torch.bfloat16, device="cuda")
    L.lsk_gemm_grouped_bf16(L.LSK_EPI_SWIGLU, xs, both, 2 * E * F, 0, F, E * F, bounds, E, h, T * k, F, H)
    y = torch.empty((T * k, H), dtype=torch.float32, device="cuda")
    L.lsk_gemm_grouped_bf16(L.LSK_EPI_SCALE_F32, h, layer.args["down"].reshape(E * H, F).contiguous(), E * H, 0, H, 0, bounds, E,
                            y, T * k, H, F, row_table=table, row_weight=w.reshape(-1))
    want = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    L.lsk_moe_combine(xd, y, T, k, H, want)
    out = layer.run(xd, lg, k)
    ref, tol = layer.reference(x, lg.cpu().numpy(), k)
    assert np.all(np.abs(to_f64(out[:T]) - to_f64(want)) <= 2 * (tol + 2.0 ** -8 * np.abs(ref)))


def test_refusals():
    layer = Layer(4, 64, 32, False, 17)
    q = Layer(4, 64, 32, True, 17)
    x = torch.zeros((80, 64), dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros((80, 4), device="cuda")
    out = torch.zeros((80, 64), dtype=torch.bfloat16, device="cuda")

    def call(layer=layer, T=2, E=4, k=2, H=64, F=32, x=x, **over):
        a = {**layer.args, **over}
        scales = {n: a[n] for n in ("gate_scales", "up_scales", "down_scales") if n in a}
        return L.lsk_moe_few(x, lg, a["gate"], a["up"], a["down"], T, E, k, H, F, out, **scales)

    def refused(status, **kw):
        with pytest.raises(L.LsError) as e:
            call(**kw)
        assert e.value.status == status

    refused(L.LS_ERR_UNSUPPORTED, T=65)
    refused(L.LS_ERR_UNSUPPORTED, E=257)
    refused(L.LS_ERR_INVALID_ARG, T=-1)
    refused(L.LS_ERR_INVALID_ARG, k=5)
    refused(L.LS_ERR_INVALID_ARG, k=0)
    refused(L.LS_ERR_INVALID_ARG, H=60)
    refused(L.LS_ERR_INVALID_ARG, F=36)
    refused(L.LS_ERR_INVALID_ARG, H=128)                      # experts closer than their bytes
    refused(L.LS_ERR_INVALID_ARG, x=x.view(-1)[1:])
    refused(L.LS_ERR_INVALID_ARG, x=None)
    refused(L.LS_ERR_INVALID_ARG, layer=q, H=1024)
    refused(L.LS_ERR_INVALID_ARG, layer=q, down=torch.zeros((5, 64, 64), dtype=torch.uint8, device="cuda").view(-1)[16:16 + 4 * 64 * 64].view(4, 64, 64))
    assert call(T=0) == L.LS_OK and call(layer=q, T=0) == L.LS_OK
    with pytest.raises(ValueError):
        call(up=Layer(4, 64, 32, False, 18, gap=1).args["up"])
