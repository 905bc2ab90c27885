"""The per-row products without a GPU: their host code linked with a runtime that launches nothing, and their binding."""
import ctypes
import os
import subprocess

import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from test_entry_host import PTR, fake_path, lib  # noqa: F401  (fixtures)

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def lora(h, epi=0, M=64, N=512, K=256, n=3, rank=16, b_rows=None, off=0, down_gap=0, up_gap=0, adapters=True, ids=PTR[2], bias=None, resid=None,
         C=PTR[4], C32=None, A=PTR[0], B=PTR[1], up2=None, down=PTR[5], up=PTR[6], scale=None):
    two = 2 if epi == L.LSK_EPI_SWIGLU else 1
    w = L.lsk_lora(n, rank, down, up, up2, scale, 2 * two * rank * K + down_gap, 2 * N * rank + up_gap)
    return h.lsk_gemm_lora_bf16(epi, A, B, N if b_rows is None else b_rows, off, ctypes.byref(w) if adapters else None, ids, bias, resid, 1, C, C32,
                                M, N, K, None)


def grouped(h, epi=0, M=64, N=100, K=256, n=5, a_rows=None, gap=0, scale_gap=0, gather_k=0, table=None, weight=None, A=PTR[0], codes=PTR[1],
            scales=PTR[2], codes2=None, scales2=None, bounds=PTR[5], C=PTR[6]):
    return h.lsk_gemm_grouped_bf16_mxfp4(epi, A, M if a_rows is None else a_rows, codes, scales, codes2, scales2,
                                         N * L.lsk_mxfp4_code_pitch(K) + gap, N * L.lsk_mxfp4_scale_pitch(K) + scale_gap, bounds, n, table, weight,
                                         gather_k, C, M, N, K, None)


CALLS = {
    "adapters, 1 row": lambda h: lora(h, M=1),
    "adapters, 17 rows": lambda h: lora(h, M=17),
    "adapters, 64 rows, gate and up": lambda h: lora(h, L.LSK_EPI_SWIGLU, off=512, b_rows=1024, up2=PTR[7]),
    "adapters, 128 rows": lambda h: lora(h, L.LSK_EPI_BIAS_RESID, M=128, bias=PTR[7], resid=PTR[8], C32=PTR[9]),
    "adapters, 1000 rows": lambda h: lora(h, L.LSK_EPI_BIAS_GELU, M=1000, bias=PTR[7]),
    "adapters, 1000 rows, gate and up": lambda h: lora(h, L.LSK_EPI_SWIGLU, M=1000, off=512, b_rows=1024, up2=PTR[7]),
    "grouped, a few rows": lambda h: grouped(h, M=20),
    "grouped, many rows": lambda h: grouped(h, L.LSK_EPI_SCALE_F32, M=5000, table=PTR[7], weight=PTR[8]),
    "grouped, gate and up": lambda h: grouped(h, L.LSK_EPI_SWIGLU, M=5000, codes2=PTR[7], scales2=PTR[8], table=PTR[9], gather_k=4, a_rows=1250),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_kernel_is_prepared_on_every_device_that_launches_it(lib, name):  # noqa: F811
    for device in (0, 1, 0, 3):
        lib.fake_set_device(device)
        before = lib.fake_launches()
        assert CALLS[name](lib) == L.LS_OK, f"refused on device {device}"
        assert lib.fake_launches() == before + 2


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_preparation_is_tried_again(lib, name):  # noqa: F811
    lib.fake_fail_allowances(1)
    assert CALLS[name](lib) == L.LS_ERR_CUDA
    assert CALLS[name](lib) == L.LS_OK
    n = lib.fake_allowances()
    assert CALLS[name](lib) == L.LS_OK and lib.fake_allowances() == n, "prepared once a device"


@pytest.mark.parametrize("M", [1, 17, 64, 128, 129, 700])
@pytest.mark.parametrize("K", [8, 1000, 11000, 1 << 20])
@pytest.mark.parametrize("rank,n", [(8, 1), (16, 64), (24, 300), (64, 4), (128, 40), (256, 500)])
def test_launches_fit_the_device(lib, M, K, rank, n):  # noqa: F811
    """Shared memory and grids of every shape's kernels: the runtime refuses what it was not asked to allow."""
    for epi, kw in ((L.LSK_EPI_STORE, {}), (L.LSK_EPI_SWIGLU, {"off": 1096, "b_rows": 2192, "up2": PTR[7]})):
        assert lora(lib, epi, M=M, N=1096, K=K, rank=rank, n=n, **kw) == L.LS_OK


BAD = L.LS_ERR_INVALID_ARG
UNS = L.LS_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    ({"epi": -1}, BAD), ({"epi": L.LSK_EPI_SCALE_F32}, BAD), ({"M": -1}, BAD), ({"N": 0}, BAD), ({"N": 12}, BAD), ({"K": 20}, BAD), ({"K": 0}, BAD),
    ({"K": (1 << 24) + 8}, BAD), ({"n": 0}, BAD), ({"rank": 0}, BAD), ({"rank": 12}, BAD), ({"rank": 264}, UNS), ({"M": 2 ** 31 - 1}, UNS),
    ({"b_rows": 511}, BAD), ({"epi": L.LSK_EPI_SWIGLU, "off": 512, "b_rows": 1023, "up2": PTR[7]}, BAD), ({"epi": L.LSK_EPI_SWIGLU, "off": 512, "b_rows": 1024}, BAD),
    ({"epi": L.LSK_EPI_BIAS_GELU}, BAD), ({"epi": L.LSK_EPI_RESID}, BAD), ({"epi": L.LSK_EPI_BIAS_RESID, "bias": PTR[7]}, BAD), ({"C32": PTR[7]}, BAD),
    ({"adapters": False}, BAD), ({"ids": None}, BAD), ({"ids": PTR[2] + 2}, BAD), ({"A": None}, BAD), ({"A": PTR[0] + 8}, BAD), ({"B": PTR[1] + 8}, BAD),
    ({"C": PTR[4] + 8}, BAD), ({"C": None}, BAD), ({"down": PTR[5] + 8}, BAD), ({"up": PTR[6] + 8}, BAD), ({"down": None}, BAD), ({"up": None}, BAD),
    ({"scale": PTR[7] + 2}, BAD), ({"down_gap": 8}, BAD), ({"up_gap": 8}, BAD), ({"down_gap": -16}, BAD), ({"up_gap": -16}, BAD),
    ({"n": 1, "down_gap": 8, "up_gap": -16}, L.LS_OK), ({"down_gap": 16, "up_gap": 32}, L.LS_OK), ({"M": 2 ** 30, "n": 512, "rank": 256}, UNS)])
def test_adapters_that_cannot_be_taken(lib, kw, status):  # noqa: F811
    assert lora(lib, **kw) == status
    if status != L.LS_OK:
        assert lib.fake_encodes() == lib.fake_pool_allocations() == lib.fake_launches() == 0


@pytest.mark.parametrize("kw,status", [
    ({"epi": L.LSK_EPI_RESID}, BAD), ({"epi": L.LSK_EPI_BIAS_GELU}, BAD), ({"M": -1}, BAD), ({"N": 0}, BAD), ({"K": 12}, BAD), ({"K": 0}, BAD),
    ({"n": 0}, BAD), ({"n": 257}, UNS), ({"M": 2 ** 30 + 1}, UNS), ({"a_rows": 63}, BAD), ({"a_rows": 63, "gather_k": 1, "table": PTR[7]}, L.LS_OK),
    ({"a_rows": 0, "gather_k": 1, "table": PTR[7]}, L.LS_OK), ({"gather_k": -1}, BAD), ({"gather_k": 2}, BAD), ({"epi": L.LSK_EPI_SCALE_F32, "table": PTR[7]}, BAD),
    ({"epi": L.LSK_EPI_SCALE_F32, "weight": PTR[7]}, BAD), ({"epi": L.LSK_EPI_SWIGLU}, BAD), ({"epi": L.LSK_EPI_SWIGLU, "codes2": PTR[7]}, BAD),
    ({"A": None}, BAD), ({"A": PTR[0] + 8}, BAD), ({"codes": PTR[1] + 16}, BAD), ({"scales": PTR[2] + 8}, BAD), ({"bounds": None}, BAD), ({"C": None}, BAD),
    ({"C": PTR[6] + 1}, BAD), ({"gap": 16}, BAD), ({"gap": 32}, L.LS_OK), ({"gap": -32}, BAD), ({"scale_gap": 8}, BAD), ({"scale_gap": 16}, L.LS_OK),
    ({"scale_gap": -16}, BAD), ({"n": 1, "gap": -32, "scale_gap": 8}, L.LS_OK), ({"N": 7}, L.LS_OK)])
def test_groups_that_cannot_be_taken(lib, kw, status):  # noqa: F811
    assert grouped(lib, **kw) == status
    if status != L.LS_OK:
        assert lib.fake_encodes() == lib.fake_pool_allocations() == lib.fake_launches() == 0


def test_no_rows_launch_nothing(lib):  # noqa: F811
    assert lora(lib, M=0, A=None, C=None) == L.LS_OK and grouped(lib, M=0, A=None, C=None) == L.LS_OK
    assert lib.fake_launches() == lib.fake_pool_allocations() == 0


# ------------------------------------------------------------------ the binding
def _adapters(n=3, r=8, N=16, K=24, two=False, **over):
    a = {"down": torch.zeros((n, r * (2 if two else 1), K), dtype=BF16), "up": torch.zeros((n, N, r), dtype=BF16),
         "up2": torch.zeros((n, N, r), dtype=BF16) if two else None, "scale": torch.zeros(n)}
    a.update(over)
    return L.lsk_lora_adapters(a["down"], a["up"], up2=a["up2"], scale=a["scale"])


def _lora(adapters=None, epi=L.LSK_EPI_STORE, N=16, K=24, **over):
    a = {"A": torch.zeros((4, K), dtype=BF16), "B": torch.zeros((2 * N, K), dtype=BF16), "ids": torch.zeros(4, dtype=I32), "C": torch.zeros((4, N), dtype=BF16)}
    kw = {k: over.pop(k) for k in ("bias", "resid", "C32") if k in over}
    a.update(over)
    return L.lsk_gemm_lora_bf16(epi, a["A"], a["B"], adapters or _adapters(), a["ids"], a["C"], 0, N, K, stream=0, **kw)


def test_adapters_are_checked_when_they_are_put_together():
    a = _adapters()
    assert (a.c.n, a.c.rank, a.c.down_stride, a.c.up_stride) == (3, 8, 2 * 8 * 24, 2 * 16 * 8)
    wide = torch.zeros((3, 8 * 24 + 16), dtype=BF16)[:, :8 * 24].unflatten(1, (8, 24))
    assert _adapters(down=wide).c.down_stride == 2 * (8 * 24 + 16)
    assert _lora() == L.LS_OK
    assert _lora(_adapters(two=True), L.LSK_EPI_SWIGLU) == L.LS_OK
    for name, t in (("down", torch.zeros((3, 8, 24))), ("up", torch.zeros((3, 16, 8), dtype=torch.float16)), ("scale", torch.zeros(3, dtype=BF16))):
        with pytest.raises(TypeError):
            _adapters(**{name: t})
    for name, t in (("down", torch.zeros((2, 8, 24), dtype=BF16)), ("down", torch.zeros((3, 16, 24), dtype=BF16)), ("up", torch.zeros((16, 8), dtype=BF16)),
                    ("up", torch.zeros((3, 8, 16), dtype=BF16).transpose(1, 2)), ("scale", torch.zeros(2)), ("scale", torch.zeros(6)[::2])):
        with pytest.raises(ValueError):
            _adapters(**{name: t})
    with pytest.raises(ValueError):
        _adapters(two=True, up2=torch.zeros((3, 17 * 8), dtype=BF16)[:, :16 * 8].unflatten(1, (16, 8)))


@pytest.mark.parametrize("name,bad,error", [
    ("A", torch.zeros((4, 24)), TypeError), ("B", torch.zeros((32, 24)), TypeError), ("C", torch.zeros((4, 16)), TypeError),
    ("ids", torch.zeros(4, dtype=torch.int64), TypeError), ("A", torch.zeros((24, 4), dtype=BF16).T, ValueError), ("ids", torch.zeros(8, dtype=I32)[::2], ValueError),
    ("C", torch.zeros((4, 32), dtype=BF16)[:, ::2], ValueError), ("bias", torch.zeros(16), TypeError), ("resid", torch.zeros((4, 16), dtype=torch.float16), TypeError),
    ("C32", torch.zeros((4, 16), dtype=BF16), TypeError)])
def test_a_product_with_adapters_takes_its_own_types(name, bad, error):
    with pytest.raises(error):
        _lora(**{name: bad})


def test_adapters_of_another_projection_are_refused():
    for kw in ({"N": 32}, {"K": 32}, {"epi": L.LSK_EPI_SWIGLU}):
        with pytest.raises(ValueError):
            _lora(**kw)
    with pytest.raises(ValueError):       # fewer ids than rows
        L.lsk_gemm_lora_bf16(0, torch.zeros((4, 24), dtype=BF16), torch.zeros((16, 24), dtype=BF16), _adapters(), torch.zeros(3, dtype=I32),
                             torch.zeros((4, 16), dtype=BF16), 4, 16, 24, stream=0)


def _grouped(epi=L.LSK_EPI_STORE, n=3, **over):
    a = {"A": torch.zeros((4, 64), dtype=BF16), "codes": torch.zeros((3, 8, 64), dtype=U8), "scales": torch.zeros((3, 8, 16), dtype=U8),
         "bounds": torch.zeros(4, dtype=I32), "C": torch.zeros((4, 8), dtype=F32 if epi == L.LSK_EPI_SCALE_F32 else BF16)}
    kw = {k: over.pop(k) for k in ("B2_codes", "B2_scales", "row_table", "row_weight") if k in over}
    a.update(over)
    return L.lsk_gemm_grouped_bf16_mxfp4(epi, a["A"], a["codes"], a["scales"], a["bounds"], n, a["C"], 0, 8, 64, stream=0, **kw)


def test_grouped_products_take_their_own_types():
    two = {"B2_codes": torch.zeros((3, 8, 64), dtype=U8), "B2_scales": torch.zeros((3, 8, 16), dtype=U8)}
    assert _grouped() == L.LS_OK and _grouped(L.LSK_EPI_SWIGLU, **two) == L.LS_OK
    assert _grouped(L.LSK_EPI_SCALE_F32, row_table=torch.zeros(4, dtype=I32), row_weight=torch.zeros(4)) == L.LS_OK
    wide = torch.zeros((3, 640), dtype=U8)[:, :512].unflatten(1, (8, 64))
    assert _grouped(codes=wide) == L.LS_OK
    for name, bad in (("A", torch.zeros((4, 64))), ("C", torch.zeros((4, 8))), ("codes", torch.zeros((3, 8, 64), dtype=BF16)),
                      ("scales", torch.zeros((3, 8, 16))), ("bounds", torch.zeros(4, dtype=torch.int64)), ("row_table", torch.zeros(4)),
                      ("row_weight", torch.zeros(4, dtype=BF16))):
        with pytest.raises(TypeError):
            _grouped(**{name: bad})
    for name, bad in (("A", torch.zeros((64, 4), dtype=BF16).T), ("codes", torch.zeros((3, 64, 8), dtype=U8).transpose(1, 2)), ("bounds", torch.zeros(3, dtype=I32)),
                      ("n", 4)):
        with pytest.raises(ValueError):
            _grouped(**{name: bad})
    with pytest.raises(ValueError):
        _grouped(L.LSK_EPI_SWIGLU, **{**two, "B2_codes": wide})


def test_adapters_are_the_headers_struct(tmp_path):
    src, exe = tmp_path / "layout.c", str(tmp_path / "layout")
    fields = [f for f, _ in L.lsk_lora._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ls_kernels.h"\nint main(void) {\n printf("%zu", sizeof(lsk_lora));\n'
                   + "".join(f' printf(" %zu", offsetof(lsk_lora, {f}));\n' for f in fields) + " return 0;\n}\n")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", include, str(src), "-o", exe], check=True)
    got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(L.lsk_lora)] + [getattr(L.lsk_lora, f).offset for f in fields]
