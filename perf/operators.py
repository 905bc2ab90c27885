"""Cases of the 4-bit and few-token operators, with their plain forms.

Four operators: writing a matrix in MXFP4 (blocks of 32 values, E2M1 elements, one power-of-two scale
each) and reading it back, the product of two MXFP4 matrices, the product of a few bf16 rows with an
MXFP4 matrix, and a whole mixture-of-experts layer for a few tokens with bf16 or MXFP4 experts.

Layout of an MXFP4 matrix [rows, K]: codes uint8 [rows, ceil(K/128)*64], two codes a byte, the even k in the
low half; scales uint8 [rows, ceil(K/32) rounded up to 16], 2^(byte - 127); padding is zero.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the activations of a small decode batch, written in 4 bits before a product
        {"name": "quantize_16x2048_bf16", "op": "quantize", "rows": 16, "K": 2048, "pad": 0, "f32": False},
        # a weight matrix of the SwiGLU stack, converted once when a model is loaded
        {"name": "quantize_13824x5120_bf16", "op": "quantize", "rows": 13824, "K": 5120, "pad": 0, "f32": False},
        # fp32 rows inside a wider buffer, K not a multiple of the block
        {"name": "quantize_1537x1000_f32_strided", "op": "quantize", "rows": 1537, "K": 1000, "pad": 24, "f32": True},
        # the up projection of the DiT stack at its 4096 tokens
        {"name": "gemm_mxfp4_4096x4096x1024", "op": "gemm", "M": 4096, "N": 4096, "K": 1024},
        # the gate projection of the SwiGLU stack over a prompt
        {"name": "gemm_mxfp4_2048x13824x5120", "op": "gemm", "M": 2048, "N": 13824, "K": 5120},
        # ragged in every direction
        {"name": "gemm_mxfp4_333x1111x1000", "op": "gemm", "M": 333, "N": 1111, "K": 1000},
        # one token through a SwiGLU gate projection
        {"name": "few_1x13824x5120", "op": "few", "M": 1, "N": 13824, "K": 5120},
        # a decode batch through the SwiGLU down projection
        {"name": "few_32x5120x13824", "op": "few", "M": 32, "N": 5120, "K": 13824},
        # a few tokens on a small ragged matrix: latency
        {"name": "few_5x1111x1000", "op": "few", "M": 5, "N": 1111, "K": 1000},
        # one token of the MoE stack's layer (128 experts, top 8), 4-bit experts: latency
        {"name": "moe_t1_mxfp4", "op": "moe", "T": 1, "E": 128, "k": 8, "H": 2048, "F": 768, "mx": True},
        # a decode batch with bf16 experts
        {"name": "moe_t16_bf16", "op": "moe", "T": 16, "E": 128, "k": 8, "H": 2048, "F": 768, "mx": False},
        # a larger decode batch with 4-bit experts
        {"name": "moe_t32_mxfp4", "op": "moe", "T": 32, "E": 128, "k": 8, "H": 2048, "F": 768, "mx": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "few", "moe"])
    while True:
        if op == "quantize":
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "K": _log_int(rng, 32, 8192),
                 "pad": rng.choice([0, 0, 1, 8, 40]), "f32": rng.random() < 0.5}
            if c["rows"] * c["K"] * (2 if c["f32"] else 1) <= 13824 * 5120:
                return c
        elif op == "gemm":
            c = {"op": op, "M": _log_int(rng, 16, 4096), "N": _log_int(rng, 64, 13824), "K": _log_int(rng, 64, 5120)}
            if c["M"] * c["N"] * c["K"] <= 2048 * 13824 * 5120:
                return c
        elif op == "few":
            c = {"op": op, "M": _log_int(rng, 1, 64), "N": _log_int(rng, 64, 13824), "K": _log_int(rng, 64, 13824)}
            if c["N"] * c["K"] <= 13824 * 5120:
                return c
        else:
            c = {"op": op, "T": _log_int(rng, 1, 64), "E": rng.randint(8, 256), "k": rng.randint(1, 8),
                 "H": 8 * _log_int(rng, 32, 512), "F": 8 * _log_int(rng, 16, 256), "mx": rng.random() < 0.5}
            if (c["E"] * c["H"] * c["F"] <= 128 * 2048 * 768 and c["T"] * c["k"] * c["H"] * c["F"] <= 32 * 8 * 2048 * 768):
                return c


# ------------------------------------------------------------------ inputs
def _normal(g, shape, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _pitches(K):
    return -(-K // 128) * 64, -(-K // 512) * 16


def _blocks(v):
    """[..., K] -> fp32 [..., 4 ceil(K/128), 32], zeros past K."""
    pad = -v.shape[-1] % 128
    v = torch.nn.functional.pad(v.float(), (0, pad)) if pad else v.float()
    return v.reshape(*v.shape[:-1], -1, 32)


def _encode(v):
    """Element codes 0..15 [..., blocks, 32] and scale exponents [..., blocks] of fp32 blocks."""
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    s = s.clamp(-127, 125)
    a = (v * ((127 - s) << 23).view(torch.float32)[..., None]).abs()   # times 2^-s, exactly
    # round to nearest, ties to the even code
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return mag + 8 * (v < 0).to(torch.uint8), s


def _pack(v):
    """MXFP4 codes and scales of [rows, K] (or [E, rows, K]) values."""
    code, s = _encode(_blocks(v))
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, -s.shape[-1] % 16))  # an empty block's byte is 0
    return byte.flatten(-2).contiguous(), scales.contiguous()


def _pack_experts(g, E, rows, K, scale):
    cp, sp = _pitches(K)
    codes = torch.empty((E, rows, cp), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, rows, sp), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (rows * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n], scales[e:e + n] = _pack(_normal(g, (n, rows, K), scale))
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2 + 1)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        R, K = case["rows"], case["K"]
        buf = _normal(g, (R, K + case["pad"]))
        buf *= torch.exp(_normal(g, (R, 1)))        # rows of different magnitude
        buf[R // 2, :min(K, 64)] = 0                # two empty blocks
        st["x"] = buf.to(torch.float32 if case["f32"] else torch.bfloat16)[:, :K]
    elif op == "gemm":
        st["a"], st["sa"] = _pack(_normal(g, (case["M"], case["K"])))
        st["b"], st["sb"] = _pack(_normal(g, (case["N"], case["K"]), case["K"] ** -0.5))
    elif op == "few":
        st["x"] = _normal(g, (case["M"], case["K"]), dtype=torch.bfloat16)
        st["b"], st["sb"] = _pack(_normal(g, (case["N"], case["K"]), case["K"] ** -0.5))
    else:
        T, E, H, F = case["T"], case["E"], case["H"], case["F"]
        st["k"] = min(case["k"], E)
        st["x"] = _normal(g, (T, H), dtype=torch.bfloat16)
        st["logits"] = _normal(g, (T, E))
        for name, rows, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
            if case["mx"]:
                st[name], st[name + "_scales"] = _pack_experts(g, E, rows, K, K ** -0.5)
            else:
                st[name] = torch.empty((E, rows, K), dtype=torch.bfloat16, device="cuda")
                for e in range(E):
                    st[name][e] = _normal(g, (rows, K), K ** -0.5)
    return st


# ------------------------------------------------------------------ the framework's operators
def _run_own(st):
    from host_offloaded_weight_gb300 import lstream as L
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["x"]
        R, K = x.shape
        codes = torch.empty((R, L.lsk_mxfp4_code_pitch(K)), dtype=torch.uint8, device="cuda")
        scales = torch.empty((R, L.lsk_mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda")
        back = torch.empty((R, K), dtype=x.dtype, device="cuda")
        L.lsk_mxfp4_quantize(x, R, K, codes, scales, ld=x.stride(0))
        L.lsk_mxfp4_dequantize(codes, scales, R, K, back)
        return back
    if op == "gemm":
        out = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
        L.lsk_gemm_mxfp4(st["a"], st["sa"], st["b"], st["sb"], out, case["M"], case["N"], case["K"])
        return out
    if op == "few":
        out = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
        L.lsk_gemm_bf16_mxfp4(st["x"], st["b"], st["sb"], out, case["M"], case["N"], case["K"])
        return out
    x = st["x"]
    out = torch.empty_like(x)
    L.lsk_moe_few(x, st["logits"], st["gate"], st["up"], st["down"], case["T"], case["E"], st["k"], case["H"], case["F"],
                  out, gate_scales=st.get("gate_scales"), up_scales=st.get("up_scales"),
                  down_scales=st.get("down_scales"))
    return out


# ------------------------------------------------------------------ plain forms, 32 bits
def _decode(codes, scales, K):
    """fp32 values [..., K] of MXFP4 codes and scales."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    blocks = codes.shape[-1] // 16
    s = (scales[..., :blocks].int() << 23).view(torch.float32)   # 2^(byte - 127) for bytes 1 to 254
    s = torch.where(scales[..., :blocks] == 0, torch.full_like(s, 2.0 ** -127), s)
    return (v.unflatten(-1, (blocks, 32)) * s[..., None]).flatten(-2)[..., :K]


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x = st["x"]
        codes, scales = _pack(x)
        return _decode(codes, scales, x.shape[1]).to(x.dtype)
    if op == "gemm":
        return (_decode(st["a"], st["sa"], case["K"]) @ _decode(st["b"], st["sb"], case["K"]).T).to(torch.bfloat16)
    if op == "few":
        return (st["x"].float() @ _decode(st["b"], st["sb"], case["K"]).T).to(torch.bfloat16)
    x = st["x"].float()
    top, sel = torch.sort(st["logits"], dim=-1, descending=True, stable=True)
    top, sel = top[:, :st["k"]], sel[:, :st["k"]]
    ex = torch.exp(top - top[:, :1])
    w = ex / ex.sum(-1, keepdim=True)

    def expert(name, K):
        if case["mx"]:
            return _decode(st[name][sel], st[name + "_scales"][sel], K)
        return st[name][sel].float()

    H, F = case["H"], case["F"]
    col = x[:, None, :, None]
    a = (expert("gate", H) @ col).squeeze(-1)
    b = (expert("up", H) @ col).squeeze(-1)
    h = a / (1.0 + torch.exp(-a)) * b
    y = (expert("down", F) @ h[..., None]).squeeze(-1)
    return (x + (w[..., None] * y).sum(1)).to(torch.bfloat16)


# ------------------------------------------------------------------ 64 bits
def _pow2(e):
    """2^e, exactly, of whole numbers e held in 64-bit floats."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_matrix(codes, scales, K):
    """Values from the format's bit fields: sign, two exponent bits (bias 1), one mantissa bit."""
    c = torch.stack((codes % 16, torch.div(codes, 16, rounding_mode="floor")), -1).flatten(-2)[..., :K].to(torch.int64)
    sign, e, m = 1.0 - 2.0 * (c // 8).double(), (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _pow2(e - 1))
    k = torch.arange(K, device=codes.device) // 32
    return sign * mag * _pow2(scales.double() - 127.0)[..., k]


def _exact_rounded(x):
    """The nearest value of the format, found among all of a block's sixteen."""
    R, K = x.shape
    out = torch.zeros((R, K), dtype=torch.float64, device=x.device)
    for k0 in range(0, K, 32):
        v = x[:, k0:k0 + 32].double()
        amax = v.abs().max(1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
        # log2 may round to a whole number next to a power of two
        e = torch.where(_pow2(e) > amax, e - 1, e)
        e = torch.where(_pow2(e + 1) <= amax, e + 1, e)
        unit = _pow2(torch.clamp(torch.where(amax > 0, e, torch.full_like(e, -125)) - 2, -127, 125))
        a = v.abs() / unit
        # steps of 1/2 below 2, of 1 below 4, of 2 above; torch.round takes ties to even
        q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
        out[:, k0:k0 + 32] = torch.sign(v) * torch.clamp(q, max=6.0) * unit
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_rounded(st["x"])
    if op == "gemm":
        b = _exact_matrix(st["b"], st["sb"], case["K"])
        return torch.cat([_exact_matrix(a, s, case["K"]) @ b.T for a, s in zip(st["a"].split(512), st["sa"].split(512))])
    if op == "few":
        x = st["x"].double()
        return torch.cat([x @ _exact_matrix(b, s, case["K"]).T for b, s in zip(st["b"].split(1024), st["sb"].split(1024))], 1)
    T, k, H, F = case["T"], st["k"], case["H"], case["F"]
    x = st["x"].double()
    y = x.clone()
    for t in range(T):
        row = st["logits"][t].double().tolist()
        order = sorted(range(case["E"]), key=lambda i: (-row[i], i))[:k]
        ws = [math.exp(row[i] - row[order[0]]) for i in order]
        for i, w in zip(order, ws):
            m = {}
            for name, K in (("gate", H), ("up", H), ("down", F)):
                m[name] = (_exact_matrix(st[name][i], st[name + "_scales"][i], K) if case["mx"] else st[name][i].double())
            a = m["gate"] @ x[t]
            y[t] += w / sum(ws) * (m["down"] @ (a * torch.sigmoid(a) * (m["up"] @ x[t])))
    return y


# ------------------------------------------------------------------ least work
def _mx_bytes(rows, K):
    return rows * K * 17 / 32


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        size = 4 if case["f32"] else 2
        # read the values, write the 4-bit form, read it and write the values that it stands for
        return {"bytes": 2 * n * size + 2 * _mx_bytes(case["rows"], case["K"]), "flops": 0}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx_bytes(M + N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "few":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx_bytes(N, K) + 2 * M * (N + K), "flops": 2 * M * N * K}
    T, E, H, F = case["T"], case["E"], case["H"], case["F"]
    k = min(case["k"], E)
    used = E * (1 - (1 - k / E) ** T)   # expected number of experts that some token is routed to
    each = _mx_bytes(3 * H * F, 1) if case["mx"] else 6 * H * F
    return {"bytes": used * each + 4 * T * H + 4 * T * E, "flops": 6 * T * k * H * F}
