"""What the binding of the grouped 4-bit products refuses because the kernel would read past its tensors."""
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L

BF16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
E, N, K, M = 3, 8, 576, 4


def _call(epi=L.LSK_EPI_STORE, rows=0, n=E, **over):
    """rows = 0 reaches the library, which launches nothing; what is refused is so before."""
    cp, sp = L.lsk_mxfp4_code_pitch(K), L.lsk_mxfp4_scale_pitch(K)
    a = {"A": torch.zeros((M, K), dtype=BF16), "codes": torch.zeros((E, N, cp), dtype=U8), "scales": torch.zeros((E, N, sp), dtype=U8),
         "row_table": torch.zeros(M, dtype=I32), "row_weight": torch.zeros(M)}
    if epi == L.LSK_EPI_SWIGLU:
        a.update(B2_codes=torch.zeros((E, N, cp), dtype=U8), B2_scales=torch.zeros((E, N, sp), dtype=U8))
    a.update(over)
    kw = {k: a[k] for k in ("B2_codes", "B2_scales", "row_table", "row_weight") if k in a}
    C = torch.zeros((M, N), dtype=torch.float32 if epi == L.LSK_EPI_SCALE_F32 else BF16)
    return L.lsk_gemm_grouped_bf16_mxfp4(epi, a["A"], a["codes"], a["scales"], torch.zeros(E + 1, dtype=I32), n, C, rows, N, K, stream=0, **kw)


def test_tensors_of_the_named_sizes_and_larger_ones_are_taken():
    cp, sp = L.lsk_mxfp4_code_pitch(K), L.lsk_mxfp4_scale_pitch(K)
    assert (cp, sp) == (320, 32)
    for epi in (L.LSK_EPI_STORE, L.LSK_EPI_SWIGLU, L.LSK_EPI_SCALE_F32):
        assert _call(epi) == L.LS_OK
    assert _call(codes=torch.zeros((E + 1, N + 2, cp), dtype=U8), scales=torch.zeros((E, N + 5, sp), dtype=U8)) == L.LS_OK
    assert _call(codes=torch.zeros((E, N * cp), dtype=U8), scales=torch.zeros((E, N * sp + 16), dtype=U8)) == L.LS_OK   # blobs
    assert _call(row_weight=torch.zeros(M + 3), A=torch.zeros((1, K), dtype=BF16)) == L.LS_OK
    assert _call(A=torch.zeros((M, 8, K // 8), dtype=BF16)) == L.LS_OK                                                    # heads side by side


@pytest.mark.parametrize("name,shape", [("codes", (E, N, 256)), ("codes", (E, N - 1, 320)), ("codes", (E, N, 384)), ("codes", (E, N * 320 - 32)),
                                        ("scales", (E, N, 16)), ("scales", (E, N - 1, 32)), ("scales", (E, N * 32 - 16)), ("B2_codes", (E, N, 256)),
                                        ("B2_scales", (E, N, 16)), ("A", (M, K - 8)), ("A", (M, K + 8)), ("A", (M * K,)), ("A", (2, 2, K))])
def test_tensors_of_other_sizes_are_refused(name, shape):
    epi = L.LSK_EPI_SWIGLU if name.startswith("B2") else L.LSK_EPI_STORE
    for n in (E, 1):       # with one group the library does not see a stride
        with pytest.raises(ValueError):
            _call(epi, n=n, **{name: torch.zeros(shape, dtype=BF16 if name == "A" else U8)})


@pytest.mark.parametrize("name,pitch", [("codes", 320), ("scales", 32), ("B2_codes", 320), ("B2_scales", 32)])
def test_a_matrix_for_each_group(name, pitch):
    epi = L.LSK_EPI_SWIGLU if name.startswith("B2") else L.LSK_EPI_STORE
    with pytest.raises(ValueError):
        _call(epi, **{name: torch.zeros((E - 1, N, pitch), dtype=U8)})
    assert _call(epi, n=E - 1, **{name: torch.zeros((E - 1, N, pitch), dtype=U8)}) == L.LS_OK
    one = torch.zeros((1, N + 4, pitch), dtype=U8)[:, :N]           # a stride that says more than there is
    with pytest.raises(ValueError):
        _call(epi, **{name: one})


def test_a_weight_for_each_row_that_the_table_may_name():
    with pytest.raises(ValueError):
        _call(L.LSK_EPI_SCALE_F32, rows=M, row_weight=torch.zeros(M - 1))
