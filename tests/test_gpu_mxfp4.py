"""The MXFP4 conversions and products against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import forward as F
from oracle import mxfp4 as mx

from gpu_util import bf16_dev, rand_bf16, to_f64

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _empty(rows, K):
    return (torch.full((rows, mx.code_pitch(K)), 0xAA, dtype=torch.uint8, device="cuda"),
            torch.full((rows, mx.scale_pitch(K)), 0xAA, dtype=torch.uint8, device="cuda"))


def _rand_mx(rows, K, seed, scale=1.0):
    """Random codes and scales on the device, and their values."""
    v = np.random.default_rng(seed).standard_normal((rows, K)) * scale
    c, s = mx.encode(v)
    return _dev(c), _dev(s), mx.decode(c, s, K)


# ------------------------------------------------------------------ conversion
QUANT = [(1, 1), (1, 32), (3, 31), (5, 33), (7, 127), (4, 128), (33, 130), (2, 511), (2, 513), (17, 1000), (300, 2048)]


def _values(rows, K, seed):
    """Values of many magnitudes, exact ties, zeros of both signs, an empty block."""
    r = np.random.default_rng(seed)
    v = r.standard_normal((rows, K)) * np.exp2(r.integers(-30, 30, (rows, 1)))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, -0.25, -5.0, 0.0, -0.0])
    v[0, :min(K, 13)] = ties[:min(K, 13)]
    if rows > 1:
        v[1, :32] = 0.0
    return v.astype(np.float32)


@pytest.mark.parametrize("rows,K", QUANT)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_quantize_and_read_back_are_the_formats(rows, K, f32, pad):
    v = _values(rows, K, rows * 1000 + K)
    t = torch.from_numpy(v)
    t = t if f32 else t.to(torch.bfloat16)
    buf = torch.full((rows, K + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :K] = t.cuda()
    codes, scales = _empty(rows, K)
    L.lsk_mxfp4_quantize(buf, rows, K, codes, scales, ld=K + pad)
    want_c, want_s = mx.encode(t.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    want = mx.decode(want_c, want_s, K)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((rows, K + pad), 77.0, dtype=dt, device="cuda")
        L.lsk_mxfp4_dequantize(codes, scales, rows, K, out, ld=K + pad)
        assert np.array_equal(out[:, :K].double().cpu().numpy(), want)
        assert bool((out[:, K:] == 77.0).all()), "wrote past K"


def test_quantize_extreme_magnitudes_and_non_finite_blocks():
    K = 32 * 9
    v = np.zeros((1, K), np.float32)
    v[0, 0:32] = np.float32(2.0 ** -149)                    # subnormal: scale byte 0
    v[0, 32:64] = np.float32(3.0e38)                        # the largest exponent
    v[0, 64:96] = np.float32(2.0 ** -126)
    v[0, 96] = np.nan
    v[0, 97:128] = 1.0
    v[0, 128] = np.inf
    v[0, 160] = -np.inf
    v[0, 192:224] = np.float32(1.5 * 2.0 ** -124)
    v[0, 224:256] = np.linspace(-8, 8, 32, dtype=np.float32)
    codes, scales = _empty(1, K)
    L.lsk_mxfp4_quantize(_dev(v), 1, K, codes, scales)
    want_c, want_s = mx.encode(v.astype(np.float64))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = torch.empty((1, K), dtype=torch.float32, device="cuda")
    L.lsk_mxfp4_dequantize(codes, scales, 1, K, back)
    got = back.cpu().numpy()
    assert np.isnan(got[0, 96:192]).all() and np.isfinite(got[0, :96]).all()
    assert np.array_equal(got.astype(np.float64), mx.decode(want_c, want_s, K), equal_nan=True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 24])
def test_a_large_matrix_has_the_bits_of_its_parts(f32, pad):
    """Large calls give a thread several rows: the last block's are not all there."""
    rows, K = 17003, 2600
    dt = torch.float32 if f32 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(41)
    src = torch.randn((rows, K + pad), generator=g, device="cuda").to(dt)
    codes, scales = _empty(rows + 1, K)
    codes[rows:], scales[rows:] = 7, 7
    L.lsk_mxfp4_quantize(src, rows, K, codes, scales, ld=K + pad)
    back = torch.full((rows, K + pad), 7.0, dtype=dt, device="cuda")
    L.lsk_mxfp4_dequantize(codes, scales, rows, K, back, ld=K + pad)
    assert bool((codes[rows:] == 7).all()) and bool((scales[rows:] == 7).all()) and bool((back[:, K:] == 7).all())
    for r0 in range(0, rows, 1000):
        n = min(1000, rows - r0)
        c, s = _empty(n, K)
        L.lsk_mxfp4_quantize(src[r0:r0 + n], n, K, c, s, ld=K + pad)
        b = torch.empty((n, K), dtype=dt, device="cuda")
        L.lsk_mxfp4_dequantize(c, s, n, K, b)
        assert torch.equal(c, codes[r0:r0 + n]) and torch.equal(s, scales[r0:r0 + n])
        assert torch.equal(b, back[r0:r0 + n, :K])


# ------------------------------------------------------------------ 4-bit x 4-bit
def _sum_tol(absum, K):
    """fp32 sums: K/32 additions, each within 2^-22 of the sum of magnitudes."""
    return (K / 32 + 8) * 2.0 ** -22 * absum


PROD = [(1, 1, 1), (1, 8, 32), (128, 192, 256), (129, 193, 257), (5, 70, 100), (300, 520, 640), (333, 1111, 1000),
        (1000, 64, 4224), (64, 4096, 128)]


@pytest.mark.parametrize("M,N,K", PROD)
@pytest.mark.parametrize("f32", [False, True])
def test_gemm_mxfp4_vs_oracle(M, N, K, f32):
    ac, as_, a = _rand_mx(M, K, 1)
    bc, bs, b = _rand_mx(N, K, 2, K ** -0.5)
    out = torch.full((M + 1, N), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    L.lsk_gemm_mxfp4(ac, as_, bc, bs, out, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    ref = a @ b.T
    tol = _sum_tol(np.abs(a) @ np.abs(b).T, K) + (0 if f32 else 2.0 ** -8 * np.abs(ref))
    assert np.all(np.abs(to_f64(out[:M]) - ref) <= tol), np.max(np.abs(to_f64(out[:M]) - ref) - tol)
    assert bool((out[M] == 77.0).all()), "wrote past the last row"


@pytest.mark.parametrize("M,N,K", [(2050, 5000, 700), (520, 10000, 260), (300, 3001, 96), (256, 17936, 1300), (1537, 1111, 2100)])
@pytest.mark.parametrize("f32", [False, True])
def test_gemm_mxfp4_many_tiles(M, N, K, f32):
    """Several tiles a CTA pair (rings and accumulators taken more than once), ragged last tiles, rows with and without alignment."""
    ac, as_, a = _rand_mx(M, K, 31)
    bc, bs, b = _rand_mx(N, K, 32, K ** -0.5)
    out = torch.full((M + 1, N), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    L.lsk_gemm_mxfp4(ac, as_, bc, bs, out, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    ref = a @ b.T
    tol = _sum_tol(np.abs(a) @ np.abs(b).T, K) + (0 if f32 else 2.0 ** -8 * np.abs(ref))
    assert np.all(np.abs(to_f64(out[:M]) - ref) <= tol)
    assert bool((out[M] == 77.0).all()), "wrote past the last row"
    again = torch.empty_like(out[:M])
    for _ in range(5):
        L.lsk_gemm_mxfp4(ac, as_, bc, bs, again, M, N, K)
        assert torch.equal(again, out[:M])



def test_gemm_mxfp4_applies_every_block_scale():
    """Each block of each row has a scale of its own, over the whole of the usual range."""
    M, N, K = 200, 260, 768
    r = np.random.default_rng(3)
    ac, as_, _ = _rand_mx(M, K, 4)
    bc, bs, _ = _rand_mx(N, K, 5)
    sa = np.zeros(as_.shape, np.uint8)
    sb = np.zeros(bs.shape, np.uint8)
    sa[:, :K // 32] = r.integers(127 - 20, 127 + 20, (M, K // 32))
    sb[:, :K // 32] = r.integers(127 - 20, 127 + 20, (N, K // 32))
    a, b = mx.decode(ac.cpu().numpy(), sa, K), mx.decode(bc.cpu().numpy(), sb, K)
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    L.lsk_gemm_mxfp4(ac, _dev(sa), bc, _dev(sb), out, M, N, K)
    assert np.all(np.abs(to_f64(out) - a @ b.T) <= _sum_tol(np.abs(a) @ np.abs(b).T, K))


def test_gemm_mxfp4_nan_blocks_stay_in_their_rows():
    M, N, K = 40, 50, 256
    ac, as_, a = _rand_mx(M, K, 6)
    bc, bs, b = _rand_mx(N, K, 7)
    as_[3, 2] = 255
    bs[11, 5] = 255
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    L.lsk_gemm_mxfp4(ac, as_, bc, bs, out, M, N, K)
    nan = np.zeros((M, N), bool)
    nan[3] = True
    nan[:, 11] = True
    assert np.array_equal(np.isnan(out.cpu().numpy()), nan)


# ------------------------------------------------------------------ bf16 x 4-bit
FEW = [(1, 1, 1), (1, 128, 128), (1, 13824, 512), (2, 200, 96), (5, 1111, 1000), (8, 300, 4096), (9, 130, 257), (16, 520, 640),
       (31, 264, 1333), (64, 700, 512), (65, 129, 384), (200, 300, 1000), (257, 640, 256)]


def _few_ref(a, b, K):
    ref = a @ b.T
    blocks = np.zeros((a.shape[0], -(-K // 32) * 32))
    blocks[:, :K] = np.abs(a)
    top = np.repeat(blocks.reshape(a.shape[0], -1, 32).max(2), 32, 1)[:, :K]
    # the sums of two terms, and what the second term leaves of values far below their block's largest
    return ref, 1.25 * _sum_tol(np.abs(a) @ np.abs(b).T, K) + 2.0 ** -21 * (top @ np.abs(b).T)


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("f32", [False, True])
def test_gemm_bf16_mxfp4_vs_oracle(M, N, K, f32):
    ab, a = rand_bf16((M, K), 11)
    bc, bs, b = _rand_mx(N, K, 12, K ** -0.5)
    out = torch.full((M + 1, N), 77.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    L.lsk_gemm_bf16_mxfp4(bf16_dev(ab), bc, bs, out, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    ref, tol = _few_ref(a, b, K)
    tol = tol + (0 if f32 else 2.0 ** -8 * np.abs(ref))
    assert np.all(np.abs(to_f64(out[:M]) - ref) <= tol), np.max(np.abs(to_f64(out[:M]) - ref) - tol)
    assert bool((out[M] == 77.0).all()), "wrote past the last row"


@pytest.mark.parametrize("M,N,K", [(3, 128 * 500, 384), (16, 128 * 470 + 60, 128), (40, 128 * 333 + 4, 640), (64, 128 * 310, 896)])
def test_gemm_bf16_mxfp4_many_tiles_of_an_odd_number_of_stages(M, N, K):
    ab, a = rand_bf16((M, K), 21)
    bc, bs, b = _rand_mx(N, K, 22, K ** -0.5)
    a_dev = bf16_dev(ab)
    outs = [torch.empty((M, N), dtype=torch.float32, device="cuda") for _ in range(5)]
    for o in outs:
        L.lsk_gemm_bf16_mxfp4(a_dev, bc, bs, o, M, N, K)
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    ref, tol = _few_ref(a, b, K)
    assert np.all(np.abs(to_f64(outs[0]) - ref) <= tol)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("pad", [1, 8])
def test_gemm_bf16_mxfp4_strided_rows_of_many_magnitudes(pad):
    M, N, K = 7, 300, 700
    r = np.random.default_rng(13)
    v = (r.standard_normal((M, K + pad)) * np.exp2(r.integers(-12, 12, (M, K + pad)))).astype(np.float32)
    t = torch.from_numpy(v).to(torch.bfloat16)
    t[:, K:] = float("nan")
    bc, bs, b = _rand_mx(N, K, 14)
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    L.lsk_gemm_bf16_mxfp4(t.cuda(), bc, bs, out, M, N, K, lda=K + pad)
    ref, tol = _few_ref(t[:, :K].double().numpy(), b, K)
    assert np.all(np.abs(to_f64(out) - ref) <= tol)


def test_gemm_bf16_mxfp4_non_finite_rows_are_nan_and_alone():
    M, N, K = 6, 150, 300
    ab, _ = rand_bf16((M, K), 15)
    t = bf16_dev(ab)
    t[2, 17] = float("nan")
    t[4, 299] = float("inf")
    bc, bs, b = _rand_mx(N, K, 16)
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    L.lsk_gemm_bf16_mxfp4(t, bc, bs, out, M, N, K)
    assert np.array_equal(np.isnan(out.cpu().numpy()).all(1), [False, False, True, False, True, False])
    assert np.isfinite(out.cpu().numpy()[[0, 1, 3, 5]]).all()


def test_products_are_the_same_bits_every_time_and_on_other_streams():
    M, N, K = 3, 5120, 2048
    ab, _ = rand_bf16((M, K), 17)
    bc, bs, _ = _rand_mx(N, K, 18)
    a = bf16_dev(ab)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(6):
        o = torch.empty((M, N), dtype=torch.float32, device="cuda")
        outs.append(o)
        L.lsk_gemm_bf16_mxfp4(a, bc, bs, o, M, N, K, stream=streams[i % 3])
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


# ------------------------------------------------------------------ refusals
def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    c, s = _empty(4, 64)
    out = torch.zeros((4, 4), dtype=torch.bfloat16, device="cuda")

    def refused(f, *a, **k):
        with pytest.raises(L.LsError) as e:
            f(*a, **k)
        assert e.value.status == L.LS_ERR_INVALID_ARG

    refused(L.lsk_mxfp4_quantize, x, 4, 64, c, s, ld=63)
    refused(L.lsk_mxfp4_quantize, x, 4, 0, c, s)
    refused(L.lsk_mxfp4_quantize, x, -1, 64, c, s)
    refused(L.lsk_mxfp4_quantize, None, 4, 64, c, s)
    refused(L.lsk_mxfp4_quantize, x, 4, 64, c.data_ptr() + 16, s)
    refused(L.lsk_mxfp4_dequantize, c, s.data_ptr() + 8, 4, 64, x)
    refused(L.lsk_gemm_mxfp4, c, s, c, s, out, 4, 0, 64)
    refused(L.lsk_gemm_mxfp4, c, s, c.data_ptr() + 16, s, out, 4, 4, 64)
    refused(L.lsk_gemm_mxfp4, c, s, c, s, None, 4, 4, 64)
    refused(L.lsk_gemm_bf16_mxfp4, x, c, s, out, 4, 4, 64, lda=60)
    refused(L.lsk_gemm_bf16_mxfp4, x, c, None, out, 4, 4, 64)
    refused(L.lsk_gemm_bf16_mxfp4, x, c, s, out, -1, 4, 64)
    for f in (lambda: L.lsk_mxfp4_quantize(x, 0, 64, c, s), lambda: L.lsk_gemm_mxfp4(c, s, c, s, out, 0, 4, 64),
              lambda: L.lsk_gemm_bf16_mxfp4(x, c, s, out, 0, 4, 64)):
        assert f() == L.LS_OK
