"""The few-token MoE layer where logits are -infinity: those experts take no part."""
import numpy as np
import pytest
import torch

from oracle import forward as F64

from gpu_util import bf16_dev, rand_bf16, to_f64
from test_gpu_moe_few import Layer

pytestmark = pytest.mark.gpu


def _poison(layer, experts):
    """The experts read as NaN (as memory that was never loaded may)."""
    for e in experts:
        for n, t in layer.args.items():
            if n.endswith("scales") or not layer.mx4:
                t[e] = 255 if layer.mx4 else float("nan")


def _reference(layer, x, lg, k, r):
    """The layer's reference and its tolerance, with the hidden activation's rounding at bf16's unit roundoff, 2^-8 of
    the value (8 significant bits, half a step): Layer.reference counts half of that."""
    ref, tol = layer.reference(x, lg, k, r)
    if not layer.mx4:
        sel, w = F64.route_topk(lg, k)
        for t in range(x.shape[0]):
            for j in range(k):
                G, U, D = (layer.values[n][sel[t, j]] for n in ("gate", "up", "down"))
                tol[t] += w[t, j] * (np.abs(D) @ (2.0 ** -9 * np.abs(F64.silu(G @ x[t]) * (U @ x[t]))))
    return ref, tol


# one and several tokens, few and many routed pairs, one CTA a tile (one pair; more tiles than SMs) and several
SHAPES = [(1, 1, 1, 64, 32), (1, 8, 4, 264, 40), (1, 128, 8, 512, 264), (2, 200, 8, 136, 72), (6, 40, 4, 128, 64),
          (9, 24, 8, 128, 64), (20, 64, 8, 264, 128), (40, 100, 6, 128, 64), (64, 256, 8, 136, 72), (3, 4, 2, 20488, 8)]


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
@pytest.mark.parametrize("mx4", [False, True])
def test_experts_behind_minus_infinity_are_left_out(T, E, k, H, F, mx4):
    """The first experts are masked for every token, all but one for the later half and all of them for some: what the
    masked experts or a token without experts hold does not matter."""
    layer = Layer(E, H, F, mx4, 3 * T + E)
    r = np.random.default_rng(T + 7 * E)
    xb, x = rand_bf16((T, H), 70)
    resid = r.standard_normal((T, H)).astype(np.float32)
    lg = r.standard_normal((T, E)).astype(np.float32)
    lg[:, :k // 2 + 1] = -np.inf
    lg[T // 2:, :E - 1] = -np.inf                # the later half has one expert
    lg[1::3] = -np.inf                           # every third token none
    none = np.isneginf(lg).all(1)
    clean = np.where(none[:, None], np.float32(0.0), lg)
    ref, tol = _reference(layer, x, clean, k, resid.astype(np.float64))
    ref[none], tol[none] = resid[none], 0.0
    _poison(layer, np.flatnonzero(np.isneginf(lg).all(0)))
    xd = bf16_dev(xb)
    xd[torch.from_numpy(none).cuda()] = float("nan")
    out32 = torch.full((T, H), 77.0, device="cuda")
    out = layer.run(xd, torch.from_numpy(lg).cuda(), k, resid=torch.from_numpy(resid).cuda(), out32=out32)
    got = to_f64(out32)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) - tol)
    assert torch.equal(out[:T], out32.to(torch.bfloat16))
    assert bool((out[T] == 77.0).all()), "wrote past the last token"


@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
@pytest.mark.parametrize("mx4", [False, True])
def test_no_token_has_an_expert(T, E, k, H, F, mx4):
    layer = Layer(E, H, F, mx4, 5)
    _poison(layer, range(E))
    xb, x = rand_bf16((T, H), 71)
    xd = bf16_dev(xb)
    out = layer.run(xd, torch.full((T, E), -np.inf, device="cuda"), k)
    assert torch.equal(out[:T], xd) and bool((out[T] == 77.0).all())


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("T", [2, 33])
def test_a_chosen_nan_beside_minus_infinity_is_nan(mx4, T):
    """NaN and -infinity are equally low: the lower index is chosen first."""
    E, k, H, F = 6, 2, 128, 64
    layer = Layer(E, H, F, mx4, 7)
    xb, x = rand_bf16((T, H), 72)
    lg = np.full((T, E), -np.inf, np.float32)
    lg[0, 1] = np.nan                            # chosen second
    lg[1, 4] = np.nan                            # not chosen: 0 and 1 are, and are left out
    xd = bf16_dev(xb)
    out = layer.run(xd, torch.from_numpy(lg).cuda(), k)
    assert bool(torch.isnan(out[0]).all()) and torch.equal(out[1:T], xd[1:])
