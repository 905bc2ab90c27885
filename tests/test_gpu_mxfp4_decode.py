"""The streamed MXFP4 MoE decode example: the same bits as with resident layers, and the oracle's values."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from oracle import forward as F64
from oracle import mxfp4 as mx

from gpu_util import to_f64

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "mxfp4_moe_decode", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_moe_decode.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def _resident(st, x):
    """The step's result with every layer on the device, in one stream."""
    logits = torch.empty((x.shape[0], st.lay.E), dtype=torch.float32, device="cuda")
    with torch.cuda.stream(st.compute):
        for blob in st.host:
            y = torch.empty_like(x)
            st.layer(blob.cuda(), x, y, logits)
            x = y
    return st.logits(x)


@pytest.mark.parametrize("layers,T", [(1, 1), (2, 5), (5, 17)])
def test_streamed_step_has_the_bits_of_resident_layers(layers, T):
    st = example.Stack(layers, 12, 264, 136, 500, 3)
    x = torch.randn((T, 264), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    torch.cuda.synchronize()
    want = _resident(st, x)
    for _ in range(3):
        got = st.step(x)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    st.check()


def test_the_head_for_few_and_many_rows_vs_oracle():
    H, V = 264, 500
    st = example.Stack(1, 4, H, 64, V, 2)
    b = mx.decode(st.head[0].cpu().numpy(), st.head[1].cpu().numpy(), H)
    for M in (3, 100):
        x = torch.randn((M, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(M)).to(torch.bfloat16)
        torch.cuda.synchronize()
        out = st.logits(x)
        torch.cuda.synchronize()
        a = to_f64(x)
        if M > example.FEW:
            a = mx.decode(*mx.encode(a), H)
        # fp32 sums of H products, and what a bf16 row's two terms leave of its blocks' largest values
        tol = 2.0 ** -20 * (np.abs(a).max() * np.abs(b).sum(1)[None] + np.abs(a) @ np.abs(b).T)
        assert np.all(np.abs(to_f64(out) - a @ b.T) <= tol)


def test_a_step_chooses_the_oracle_s_experts():
    """One layer's output against the 64-bit layer on the values that the codes stand for."""
    E, H, F, k, T = 6, 128, 64, 2, 4
    st = example.Stack(1, E, H, F, 64, k)
    blob = st.host[0]

    def values(name, rows, K):
        c, s = (st.lay.view(blob, name, p).numpy() for p in ("codes", "scales"))
        return mx.decode(c, s, K).reshape(-1, rows, K)

    R, G, U, D = values("router", E, H)[0], values("gate", F, H), values("up", F, H), values("down", H, F)
    x = torch.randn((T, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(torch.bfloat16)
    torch.cuda.synchronize()
    out, logits = torch.empty_like(x), torch.empty((T, E), dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    st.layer(blob.cuda(), x, out, logits)
    torch.cuda.synchronize()
    xv = to_f64(x)
    assert np.max(np.abs(to_f64(logits) - xv @ R.T)) < 1e-4
    sel, w = F64.route_topk(logits.cpu().numpy(), k)
    want = xv.copy()
    for t in range(T):
        for j in range(k):
            e = sel[t, j]
            want[t] += w[t, j] * (D[e] @ (F64.silu(G[e] @ xv[t]) * (U[e] @ xv[t])))
    assert np.max(np.abs(to_f64(out) - want)) <= 1e-2 * np.max(np.abs(want))


def test_main_runs():
    assert example.main(["--layers", "3", "--experts", "8", "--hidden", "256", "--ffn", "128", "--vocab", "1000", "--top-k", "2",
                         "--tokens", "2", "--prompt", "80", "--steps", "2"]) == 0
    assert L.lsk_device_error() == 0
