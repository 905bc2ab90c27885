"""bf16 rows beside MXFP4 weights at both ends of the exponent range, in each of the product's row paths."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import forward as F64
from oracle import mxfp4 as mx

from gpu_util import bf16_dev, to_f64
from test_gpu_moe_few import Layer
from test_gpu_mxfp4 import _dev, _few_ref

pytestmark = pytest.mark.gpu

ROWS = [3, 8, 12, 40, 130]       # up to 8 rows are split on their way into the product, more by a kernel before it


def _rows(M, K, lo, hi, seed):
    """bf16 bits and values with exponent fields lo to hi: blocks of one magnitude and of many, the largest mantissas."""
    r = np.random.default_rng(seed)
    field = r.integers(lo, hi + 1, (M, K))
    block = r.integers(lo, hi + 1, (M, -(-K // 32))).repeat(32, 1)[:, :K]
    field = np.where(r.random((M, 1)) < 0.5, block, field)
    mant = np.where(r.random((M, K)) < 0.3, r.integers(0x78, 0x80, (M, K)), r.integers(0, 0x80, (M, K)))
    bits = (r.integers(0, 2, (M, K)) << 15 | field << 7 | mant).astype(np.uint16)
    return bits, F64.bf16_bits_to_f64(bits)


def _product(bits, codes, scales, N, K):
    M = bits.shape[0]
    out = torch.full((M + 1, N), 77.0, device="cuda")
    L.lsk_gemm_bf16_mxfp4(bf16_dev(bits), codes, scales, out, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    assert bool((out[M] == 77.0).all()), "wrote past the last row"
    return to_f64(out[:M])


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("lo,hi,w", [(0, 12, 2.0 ** 40), (0, 0, 2.0 ** 40), (110, 140, 1.0), (245, 254, 2.0 ** -40),
                                     (254, 254, 2.0 ** -40)])
def test_products_of_the_smallest_and_the_largest_rows(M, lo, hi, w):
    """Subnormal rows, rows next to the largest number; weights that bring the results back to ordinary size."""
    N, K = 200, 328
    bits, a = _rows(M, K, lo, hi, M + lo)
    c, s = mx.encode(np.random.default_rng(lo).standard_normal((N, K)) * w)
    ref, tol = _few_ref(a, mx.decode(c, s, K), K)
    got = _product(bits, _dev(c), _dev(s), N, K)
    assert np.all(np.abs(got - ref) <= tol), np.max((np.abs(got - ref) - tol) / np.abs(ref).max())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("lo,hi", [(14, 27), (120, 133), (241, 254), (254, 254)])
def test_every_value_down_to_a_8192th_of_its_block_comes_through_whole(M, lo, hi):
    """Unit rows of weights give A back; the exponents span 2^13, so all eight bits of each value are kept."""
    K = 96
    bits, a = _rows(M, K, lo, hi, M + hi)
    c, s = mx.encode(np.eye(K))
    assert np.array_equal(_product(bits, _dev(c), _dev(s), K, K), a)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("M", [12, 40, 130])
def test_many_strided_rows_of_many_magnitudes(M, pad):
    N, K = 300, 700
    r = np.random.default_rng(13 + M)
    v = (r.standard_normal((M, K + pad)) * np.exp2(r.integers(-12, 12, (M, K + pad)))).astype(np.float32)
    t = torch.from_numpy(v).to(torch.bfloat16)
    t[:, K:] = float("nan")
    c, s = mx.encode(r.standard_normal((N, K)))
    out = torch.empty((M, N), device="cuda")
    L.lsk_gemm_bf16_mxfp4(t.cuda(), _dev(c), _dev(s), out, M, N, K, lda=K + pad)
    ref, tol = _few_ref(t[:, :K].double().numpy(), mx.decode(c, s, K), K)
    assert np.all(np.abs(to_f64(out) - ref) <= tol)


@pytest.mark.parametrize("M", [12, 40, 130])
def test_many_rows_with_non_finite_ones_among_them(M):
    N, K = 150, 300
    r = np.random.default_rng(M)
    t = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    t[2, 17] = float("nan")
    t[4, 299] = float("inf")
    t[M - 1, 0] = float("-inf")
    c, s = mx.encode(r.standard_normal((N, K)))
    out = torch.empty((M, N), device="cuda")
    L.lsk_gemm_bf16_mxfp4(t, _dev(c), _dev(s), out, M, N, K)
    bad = np.zeros(M, bool)
    bad[[2, 4, M - 1]] = True
    got = out.cpu().numpy()
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("mant", [255, 254, 249, 248, 247, 129, 128])
@pytest.mark.parametrize("back", [0, -100])
def test_hidden_activations_next_to_the_largest_number(T, mant, back):
    """h = mant 2^120 in every column of every token; one column of h for each row of down, times 2^back."""
    H, F = 256, 64
    layer = Layer(1, H, F, True, 9)
    for name, rows, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
        w = np.zeros((rows, K))
        if name == "down":
            w[:F] = np.eye(F) * 2.0 ** back
        else:
            w[:, 0 if name == "gate" else 64] = 1.0
        c, s = mx.encode(w)
        layer.args[name] = _dev(c)[None]
        layer.args[name + "_scales"] = _dev(s)[None]
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    x[:, 0] = 2.0 ** 60                          # the gate: SiLU of it is itself
    x[:, 64] = float(mant) * 2.0 ** 60           # the other factor
    out32 = torch.empty((T, H), device="cuda")
    layer.run(x.cuda(), torch.zeros((T, 1), device="cuda"), 1, resid=torch.zeros((T, H), device="cuda"), out32=out32)
    want = np.zeros((T, H))
    want[:, :F] = mant * 2.0 ** (120 + back)
    assert np.array_equal(to_f64(out32), want)
