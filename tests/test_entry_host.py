"""The kernels' host code without a GPU: the library's own objects linked with a runtime of two devices that launches
nothing (abi/fake_runtime.c)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from host_offloaded_weight_gb300 import build as B
from host_offloaded_weight_gb300 import lstream as L

HERE = os.path.dirname(os.path.abspath(__file__))
LEFT_OUT = ("runtime.cu", "ls_sched.cpp", "kapi_static.cu")   # the streaming runtime


def _undefined(path):
    out = subprocess.run(["nm", "-u", path], capture_output=True, text=True, check=True).stdout
    return {ln.split()[-1] for ln in out.splitlines()}


@pytest.fixture(scope="module")
def fake_path(tmp_path_factory):
    B.build()          # the objects, where they are older than their sources
    d = tmp_path_factory.mktemp("fake")
    objs = [os.path.join(B.BUILD, os.path.splitext(s)[0] + ".o") for s in B.SOURCES if s not in LEFT_OUT]
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B._nvcc()))), "include")
    fake, rest, lib = str(d / "fake.o"), str(d / "rest.c"), str(d / "libfake.so")
    subprocess.run(["gcc", "-O1", "-fPIC", "-Wall", "-Werror", "-I", include, "-c", os.path.join(HERE, "abi", "fake_runtime.c"),
                    "-o", fake], check=True)
    has = subprocess.run(["nm", "--defined-only", fake], capture_output=True, text=True, check=True).stdout
    has = {ln.split()[-1] for ln in has.splitlines()}
    missing = sorted(s for s in set().union(*map(_undefined, objs)) - has if s.startswith("cuda"))
    with open(rest, "w") as f:
        f.writelines(f"int {s}(void) {{ return 801; }}\n" for s in missing)   # cudaErrorNotSupported
    subprocess.run(["g++", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-o", lib, *objs, fake, "-x", "c", rest], check=True)
    return lib


@pytest.fixture
def lib(fake_path, tmp_path):
    """A copy of its own for each test: nothing is known of any device yet."""
    path = str(tmp_path / "libfake.so")
    shutil.copy(fake_path, path)
    h = ctypes.CDLL(path)
    for name, (res, args) in L._sig.items():
        f = getattr(h, name, None)
        if f is not None:
            f.restype, f.argtypes = res, args
    return h


PTR = [(i + 1) << 32 for i in range(12)]      # aligned, apart, never read


def experts(mx, E, H, F, gap=0, scale_gap=0, down_gap=0):
    up = F * (L.lsk_mxfp4_code_pitch(H) if mx else 2 * H) + gap
    down = H * (L.lsk_mxfp4_code_pitch(F) if mx else 2 * F) + down_gap
    return L.lsk_moe_experts(int(mx), 0, PTR[0], PTR[1], PTR[2], up, down, PTR[3], PTR[4], PTR[5],
                             F * L.lsk_mxfp4_scale_pitch(H) + scale_gap, H * L.lsk_mxfp4_scale_pitch(F) + scale_gap)


def moe(h, mx, T=4, E=8, k=2, H=128, F=64, **gaps):
    w = experts(mx, E, H, F, **gaps)
    return h.lsk_moe_few(PTR[6], None, PTR[7], ctypes.byref(w), T, E, k, H, F, PTR[8], None, None)


CALLS = {
    "4-bit product, narrow tiles": lambda h: h.lsk_gemm_mxfp4(*PTR[:5], 0, 100, 64, 500, None),
    "4-bit product, wide tiles": lambda h: h.lsk_gemm_mxfp4(*PTR[:5], 1, 4096, 4096, 1024, None),
    "bf16 x 4-bit, 3 rows": lambda h: h.lsk_gemm_bf16_mxfp4(PTR[0], 256, PTR[1], PTR[2], PTR[3], 0, 3, 512, 256, None),
    "bf16 x 4-bit, 16 rows": lambda h: h.lsk_gemm_bf16_mxfp4(PTR[0], 256, PTR[1], PTR[2], PTR[3], 0, 16, 512, 256, None),
    "bf16 x 4-bit, 32 rows": lambda h: h.lsk_gemm_bf16_mxfp4(PTR[0], 256, PTR[1], PTR[2], PTR[3], 0, 32, 512, 256, None),
    "bf16 x 4-bit, 64 rows": lambda h: h.lsk_gemm_bf16_mxfp4(PTR[0], 256, PTR[1], PTR[2], PTR[3], 0, 64, 512, 256, None),
    "bf16 x 4-bit, 300 rows": lambda h: h.lsk_gemm_bf16_mxfp4(PTR[0], 256, PTR[1], PTR[2], PTR[3], 0, 300, 512, 256, None),
    "MoE layer, bf16": lambda h: moe(h, False),
    "MoE layer, MXFP4": lambda h: moe(h, True),
    "dense product": lambda h: h.lsk_gemm_bf16(0, PTR[0], PTR[1], 512, 0, PTR[3], None, 0, PTR[2], None, 512, 512, 256, 0, None),
    "dense product of few rows": lambda h: h.lsk_gemm_bf16(0, PTR[0], PTR[1], 4096, 0, PTR[3], None, 0, PTR[2], None, 64, 4096, 256, 0,
                                                           None),
    "fp32 linear": lambda h: h.lsk_linear_gelu_f32(PTR[0], PTR[1], PTR[2], PTR[3], 4, 2048, 256, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_kernel_is_prepared_on_every_device_that_launches_it(lib, name):
    for device in (0, 1, 0, 3):
        lib.fake_set_device(device)
        before = lib.fake_launches()
        assert CALLS[name](lib) == L.LS_OK, f"refused on device {device}"
        assert lib.fake_launches() > before


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_preparation_is_tried_again(lib, name):
    lib.fake_fail_allowances(1)
    assert CALLS[name](lib) == L.LS_ERR_CUDA
    assert CALLS[name](lib) == L.LS_OK
    n = lib.fake_allowances()
    assert CALLS[name](lib) == L.LS_OK and lib.fake_allowances() == n, "prepared once a device"


def test_a_larger_need_is_asked_for_and_a_smaller_one_is_not(lib):
    def linear(H):
        return lib.lsk_linear_gelu_f32(PTR[0], PTR[1], PTR[2], PTR[3], 4, H, 256, None)

    asked = []
    for device in (0, 1):
        lib.fake_set_device(device)
        for H in (1024, 2048, 1024, 2048):
            n = lib.fake_allowances()
            assert linear(H) == L.LS_OK
            asked.append(lib.fake_allowances() - n)
    assert asked == [1, 1, 0, 0] * 2


def test_grids_are_sized_for_the_current_device(lib):
    for device, sms in ((1, 76), (0, 152), (2, 76)):
        lib.fake_set_device(device)
        assert lib.lsk_num_sms() == sms
        assert CALLS["4-bit product, wide tiles"](lib) == L.LS_OK and lib.fake_last_grid() <= sms


@pytest.mark.parametrize("mx,gaps,status", [
    (True, {"gap": 32}, L.LS_OK), (True, {"down_gap": 96}, L.LS_OK), (True, {"scale_gap": 16}, L.LS_OK),
    (True, {"gap": 16}, L.LS_ERR_INVALID_ARG), (True, {"down_gap": 48}, L.LS_ERR_INVALID_ARG),
    (True, {"scale_gap": 8}, L.LS_ERR_INVALID_ARG), (True, {"gap": -32}, L.LS_ERR_INVALID_ARG),
    (False, {"gap": 16}, L.LS_OK), (False, {"down_gap": 48}, L.LS_OK), (False, {"gap": 8}, L.LS_ERR_INVALID_ARG),
    (False, {"down_gap": -16}, L.LS_ERR_INVALID_ARG)])
def test_strides_between_experts(lib, mx, gaps, status):
    """Packed codes are unpacked by tensor copies whose strides are multiples of 32 bytes: refused as arguments, before
    scratch is taken or a tensor map is made."""
    assert moe(lib, mx, **gaps) == status
    if status != L.LS_OK:
        assert lib.fake_encodes() == lib.fake_pool_allocations() == lib.fake_launches() == 0
    assert moe(lib, mx, E=1, k=1, **gaps) == L.LS_OK, "one expert's strides are not read"


@pytest.mark.parametrize("M,N,status", [
    (2 ** 31 - 256, 8, L.LS_OK), (8, 2 ** 31 - 224, L.LS_OK), (2 ** 31 - 255, 8, L.LS_ERR_UNSUPPORTED),
    (8, 2 ** 31 - 223, L.LS_ERR_UNSUPPORTED), (2 ** 31 - 1, 8, L.LS_ERR_UNSUPPORTED), (8, 2 ** 31 - 1, L.LS_ERR_UNSUPPORTED)])
def test_rows_of_the_4_bit_product_stay_below_the_limit(lib, M, N, status):
    """Tiles of 256 rows and 224 columns are counted in 32 bits."""
    assert lib.lsk_gemm_mxfp4(*PTR[:5], 0, M, N, 32, None) == status
    assert lib.fake_launches() == (status == L.LS_OK)


@pytest.mark.parametrize("M,N,status", [(2 ** 30 - 128, 8, L.LS_OK), (2 ** 30 - 127, 8, L.LS_ERR_UNSUPPORTED),
                                        (3, 2 ** 31 - 1, L.LS_OK)])
def test_rows_of_the_bf16_product_stay_below_the_limit(lib, M, N, status):
    assert lib.lsk_gemm_bf16_mxfp4(PTR[0], 32, PTR[1], PTR[2], PTR[3], 0, M, N, 32, None) == status
    assert (lib.fake_launches() > 0) == (status == L.LS_OK)
