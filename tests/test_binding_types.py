"""The 4-bit operators' binding: types and layouts that the kernels would read wrongly are errors before any launch."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
E, H, F = 3, 64, 32


def _moe(mx=False, **over):
    """A call for no token at all: the library returns before it needs a device."""
    pitch, spitch = L.lsk_mxfp4_code_pitch, L.lsk_mxfp4_scale_pitch
    a = {"x": torch.zeros((2, H), dtype=BF16), "logits": torch.zeros((2, E)), "out": torch.zeros((2, H), dtype=BF16)}
    for name, rows, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
        a[name] = torch.zeros((E, rows, pitch(K)), dtype=U8) if mx else torch.zeros((E, rows, K), dtype=BF16)
        if mx:
            a[name + "_scales"] = torch.zeros((E, rows, spitch(K)), dtype=U8)
    a.update(over)
    return L.lsk_moe_few(a.pop("x"), a.pop("logits"), a.pop("gate"), a.pop("up"), a.pop("down"), 0, E, 2, H, F, a.pop("out"),
                         stream=0, **a)


def _product(A=None, out=None, codes=None, scales=None, **kw):
    A = torch.zeros((4, 64), dtype=BF16) if A is None else A
    out = torch.zeros((4, 8), dtype=BF16) if out is None else out
    codes = torch.zeros((8, 64), dtype=U8) if codes is None else codes
    scales = torch.zeros((8, 16), dtype=U8) if scales is None else scales
    return L.lsk_gemm_bf16_mxfp4(A, codes, scales, out, 0, 8, 64, stream=0, **kw)


@pytest.mark.parametrize("mx", [False, True])
def test_moe_layer_takes_its_own_types(mx):
    assert _moe(mx) == L.LS_OK
    assert _moe(mx, resid=torch.zeros((2, H)), out32=torch.zeros((2, H))) == L.LS_OK
    assert _moe(mx, x=4096, out=4096, logits=4096) == L.LS_OK, "raw addresses pass"
    wide = torch.zeros((E, 40 * 64), dtype=U8 if mx else BF16)[:, :F * 64]      # experts apart
    assert _moe(mx, gate=wide.unflatten(1, (F, 64)), up=wide.unflatten(1, (F, 64))) == L.LS_OK


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("name,bad", [
    ("x", F32), ("x", torch.float16), ("out", F32), ("logits", BF16), ("logits", torch.float64), ("resid", BF16), ("out32", BF16),
    ("gate", F32), ("up", F32), ("down", F32), ("down", torch.float16)])
def test_moe_layer_refuses_other_types(mx, name, bad):
    shapes = {"logits": (2, E), "gate": (E, F, H), "up": (E, F, H), "down": (E, H, F)}
    with pytest.raises(TypeError):
        _moe(mx, **{name: torch.zeros(shapes.get(name, (2, H)), dtype=bad)})


def test_codes_need_their_scales_and_scales_are_bytes():
    codes = torch.zeros((E, F, 64), dtype=U8)
    with pytest.raises(TypeError):
        _moe(False, gate=codes)
    for name, rows in (("gate", F), ("up", F), ("down", H)):
        with pytest.raises(TypeError):
            _moe(True, **{name + "_scales": torch.zeros((E, rows, 16))})


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("name", ["x", "logits", "out", "resid", "out32", "gate", "down"])
def test_moe_layer_refuses_other_layouts(mx, name):
    if name in ("gate", "down"):
        rows, cols = (F, 64) if name == "gate" else (H, 64 if mx else F)
        t = torch.zeros((E, rows, cols + 8), dtype=U8 if mx else BF16)[:, :, :cols]
    else:
        dt = F32 if name in ("logits", "resid", "out32") else BF16
        n = E if name == "logits" else H
        t = torch.zeros((2, n + 8), dtype=dt)[:, :n]
    with pytest.raises(ValueError):
        _moe(mx, **{name: t})


def test_bf16_product():
    assert _product() == L.LS_OK and _product(out=torch.zeros((4, 8))) == L.LS_OK
    wide = torch.zeros((4, 80), dtype=BF16)[:, :64]
    assert _product(wide, lda=80) == L.LS_OK
    for A in (torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.float16), torch.zeros((4, 64), dtype=torch.float64)):
        with pytest.raises(TypeError):
            _product(A)
    for kw in ({"A": wide}, {"A": torch.zeros((64, 4), dtype=BF16).T, "lda": 64}, {"out": torch.zeros((4, 16))[:, :8]},
               {"codes": torch.zeros((8, 80), dtype=U8)[:, :64]}, {"scales": torch.zeros((8, 32), dtype=U8)[:, :16]}):
        with pytest.raises(ValueError):
            _product(**kw)
    for kw in ({"codes": torch.zeros((8, 64), dtype=torch.int32)}, {"scales": torch.zeros((8, 16))}):
        with pytest.raises(TypeError):
            _product(**kw)


def test_conversions_and_the_4_bit_product():
    codes, scales = torch.zeros((4, 64), dtype=U8), torch.zeros((4, 16), dtype=U8)
    x, wide = torch.zeros((4, 64)), torch.zeros((4, 80))[:, :64]
    for f in (lambda t, **k: L.lsk_mxfp4_quantize(t, 0, 64, codes, scales, stream=0, **k),
              lambda t, **k: L.lsk_mxfp4_dequantize(codes, scales, 0, 64, t, stream=0, **k)):
        assert f(x) == L.LS_OK and f(wide, ld=80) == L.LS_OK and f(np.zeros((4, 64), np.float32)) == L.LS_OK
        with pytest.raises(ValueError):
            f(wide)
        with pytest.raises(ValueError):
            f(torch.zeros((64, 4)).T, ld=64)
        with pytest.raises(TypeError):
            f(x.half())
    out = torch.zeros((4, 4))
    assert L.lsk_gemm_mxfp4(codes, scales, codes, scales, out, 0, 4, 64, stream=0) == L.LS_OK
    with pytest.raises(TypeError):
        L.lsk_gemm_mxfp4(codes.int(), scales, codes, scales, out, 0, 4, 64, stream=0)
    with pytest.raises(ValueError):
        L.lsk_gemm_mxfp4(codes, scales, codes, scales, torch.zeros((4, 8))[:, :4], 0, 4, 64, stream=0)


def test_packed_experts_are_the_headers_struct(tmp_path):
    import ctypes
    import os
    import subprocess
    v = [1, 0] + [(i + 1) << 33 for i in range(10)]
    assert L._experts(*v) == bytes(L.lsk_moe_experts(*v))
    src = tmp_path / "layout.c"
    fields = [f for f, _ in L.lsk_moe_experts._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ls_kernels.h"\nint main(void) {\n printf("%zu", sizeof(lsk_moe_experts));\n'
                   + "".join(f' printf(" %zu", offsetof(lsk_moe_experts, {f}));\n' for f in fields) + " return 0;\n}\n")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", include, str(src), "-o", exe], check=True)
    got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(L.lsk_moe_experts)] + [getattr(L.lsk_moe_experts, f).offset for f in fields]


@pytest.mark.parametrize("mx", [False, True])
def test_one_experts_strides_are_free(mx):
    """A layer of one expert, its matrices cut out of stacks of different kinds."""
    def cut(rows, cols, gap, dt):
        return torch.zeros((2, rows + gap, cols), dtype=dt)[:1, :rows]

    dt, pitch = (U8, L.lsk_mxfp4_code_pitch) if mx else (BF16, lambda K: K)
    x, out, lg = torch.zeros((2, H), dtype=BF16), torch.zeros((2, H), dtype=BF16), torch.zeros((2, 1))
    scales = {n + "_scales": cut(rows, 16, i, U8) for i, (n, rows) in enumerate((("gate", F), ("up", F), ("down", H)))} if mx else {}
    assert L.lsk_moe_few(x, lg, cut(F, pitch(H), 3, dt), cut(F, pitch(H), 0, dt), cut(H, pitch(F), 1, dt), 0, 1, 1, H, F, out,
                         stream=0, **scales) == L.LS_OK
