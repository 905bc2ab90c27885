"""Calls in flight on several streams at once: each has its scratch to itself."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import mxfp4 as mx

from gpu_util import bf16_dev, rand_bf16
from test_gpu_moe_few import Layer
from test_gpu_mxfp4 import _rand_mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 12, 40, 200])
def test_products_of_different_inputs_in_flight_on_three_streams(M):
    N, K, calls = 2000, 2176, 24
    bc, bs, _ = _rand_mx(N, K, 1)
    xs = [bf16_dev(rand_bf16((M, K), 10 + i)[0]) for i in range(4)]
    want = []
    for x in xs:
        o = torch.empty((M, N), device="cuda")
        L.lsk_gemm_bf16_mxfp4(x, bc, bs, o, M, N, K)
        torch.cuda.synchronize()
        want.append(o)
    outs = [torch.empty((M, N), device="cuda") for _ in range(calls)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        L.lsk_gemm_bf16_mxfp4(xs[i % 4], bc, bs, o, M, N, K, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 4])


@pytest.mark.parametrize("M", [5, 12, 300])
def test_quantised_weights_are_complete_before_the_product_behind_them_reads(M):
    """Conversion and product alternate on one stream, over the same buffers."""
    N, K = 1500, 1408
    ws = [bf16_dev(rand_bf16((N, K), 30 + i)[0]) for i in range(3)]
    x = bf16_dev(rand_bf16((M, K), 40)[0])
    codes = torch.empty((N, mx.code_pitch(K)), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, mx.scale_pitch(K)), dtype=torch.uint8, device="cuda")
    want = []
    for w in ws:
        o = torch.empty((M, N), device="cuda")
        L.lsk_mxfp4_quantize(w, N, K, codes, scales)
        torch.cuda.synchronize()
        L.lsk_gemm_bf16_mxfp4(x, codes, scales, o, M, N, K)
        torch.cuda.synchronize()
        want.append(o)
    outs = [torch.empty((M, N), device="cuda") for _ in range(12)]
    for i, o in enumerate(outs):
        L.lsk_mxfp4_quantize(ws[i % 3], N, K, codes, scales)
        L.lsk_gemm_bf16_mxfp4(x, codes, scales, o, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 3])


@pytest.mark.parametrize("mx4", [False, True])
def test_moe_layers_of_different_inputs_in_flight_on_three_streams(mx4):
    E, k, H, F = 24, 4, 520, 264
    layer = Layer(E, H, F, mx4, 21)
    cases = []
    for i, T in enumerate((1, 12, 40)):
        x = bf16_dev(rand_bf16((T, H), 50 + i)[0])
        lg = torch.from_numpy(np.random.default_rng(60 + i).standard_normal((T, E)).astype(np.float32)).cuda()
        cases.append((T, x, lg, layer.run(x, lg, k)[:T].clone()))
    a = layer.args
    scales = {n: a[n] for n in ("gate_scales", "up_scales", "down_scales") if n in a}
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.zeros_like(cases[i % 3][3]) for i in range(18)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        T, x, lg, _ = cases[i % 3]
        L.lsk_moe_few(x, lg, a["gate"], a["up"], a["down"], T, E, k, H, F, o, stream=streams[(i // 2) % 3], **scales)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, cases[i % 3][3])


@pytest.mark.parametrize("M", [1, 12, 40, 200])
def test_conversion_and_products_in_a_graph(M):
    """Weights converted, read back and multiplied in one captured chain; the inputs change between replays."""
    N, K = 900, 1400
    w = torch.empty((N, K), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    codes, xcodes = (torch.empty((r, mx.code_pitch(K)), dtype=torch.uint8, device="cuda") for r in (N, M))
    scales, xscales = (torch.empty((r, mx.scale_pitch(K)), dtype=torch.uint8, device="cuda") for r in (N, M))
    back = torch.empty_like(w)
    out, out4 = torch.empty((M, N), device="cuda"), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")

    def chain():
        L.lsk_mxfp4_quantize(w, N, K, codes, scales)
        L.lsk_gemm_bf16_mxfp4(x, codes, scales, out, M, N, K)
        L.lsk_mxfp4_quantize(x, M, K, xcodes, xscales)
        L.lsk_gemm_mxfp4(xcodes, xscales, codes, scales, out4, M, N, K)
        L.lsk_mxfp4_dequantize(codes, scales, N, K, back)

    def fill(i):
        w.copy_(bf16_dev(rand_bf16((N, K), 70 + i)[0]))
        x.copy_(bf16_dev(rand_bf16((M, K), 80 + i)[0]))

    want = []
    for i in range(3):
        fill(i)
        chain()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (out, out4, back)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for i in (0, 1, 2, 0):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        for got, ref in zip((out, out4, back), want[i]):
            assert torch.equal(got, ref)
