"""Cases of the products whose weights differ by rows, with their plain forms.

Two operators: a projection shared by all requests with each request's own low-rank adapter beside it, and the
products of a mixture of MXFP4 experts for any number of tokens, grouped by expert with ragged group sizes.

Adapters: row t with adapter a = ids[t] gets  s_a up_a (down_a x_t)  added to its shared product W x_t, before the
bias, the residual or the activation; a negative id is no adapter. Experts: the row i of the sorted order belongs to
the group that bounds say and to row table[i] = t k + j of the routing; the first product gives SiLU(G_e x) * (U_e x),
the second one the rows weight[table[i]] D_e h_i at their places table[i].

Layout of an MXFP4 matrix [rows, K]: codes uint8 [rows, ceil(K/128)*64], two codes a byte, the even k in the
low half; scales uint8 [rows, ceil(K/32) rounded up to 16], 2^(byte - 127); padding is zero.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one row through the DiT stack's up projection, a small adapter beside it: latency
        {"name": "lora_1x4096x1024_gelu_r8", "op": "lora", "T": 1, "N": 4096, "K": 1024, "r": 8, "n": 4, "reqs": 1, "epi": "gelu"},
        # a decode batch through the SwiGLU stack's gate projection, every request with an adapter of its own
        {"name": "lora_16x13824x5120_r16", "op": "lora", "T": 16, "N": 13824, "K": 5120, "r": 16, "n": 64, "reqs": 16, "epi": "store"},
        # a larger decode batch through the down projection, with bias and the fp32 residual stream
        {"name": "lora_64x5120x13824_resid_r32", "op": "lora", "T": 64, "N": 5120, "K": 13824, "r": 32, "n": 24, "reqs": 64, "epi": "resid"},
        # ragged in every direction, a few drafted tokens of some requests
        {"name": "lora_37x1096x1000_r24", "op": "lora", "T": 37, "N": 1096, "K": 1000, "r": 24, "n": 8, "reqs": 9, "epi": "store"},
        # the DiT stack's 4096 tokens of four requests
        {"name": "lora_4096x4096x1024_gelu_r64", "op": "lora", "T": 4096, "N": 4096, "K": 1024, "r": 64, "n": 4, "reqs": 4, "epi": "gelu"},
        # prompts of several requests through the SwiGLU stack's gate and up projections
        {"name": "lora_2048x13824x5120_swiglu_r16", "op": "lora", "T": 2048, "N": 13824, "K": 5120, "r": 16, "n": 16, "reqs": 7, "epi": "swiglu"},
        # one token of the MoE stack's layer: eight experts with a row each, latency
        {"name": "experts_up_t1", "op": "up", "T": 1, "E": 128, "k": 8, "H": 2048, "F": 768, "skew": 0.0},
        # a decode batch larger than the few-token layer takes, experts of a few rows
        {"name": "experts_up_t96", "op": "up", "T": 96, "E": 128, "k": 8, "H": 2048, "F": 768, "skew": 0.5},
        {"name": "experts_down_t512", "op": "down", "T": 512, "E": 128, "k": 8, "H": 2048, "F": 768, "skew": 0.5},
        # ragged sizes, some experts without a row
        {"name": "experts_down_t333_ragged", "op": "down", "T": 333, "E": 40, "k": 3, "H": 1000, "F": 712, "skew": 2.0},
        # a long prompt
        {"name": "experts_up_t4096", "op": "up", "T": 4096, "E": 128, "k": 8, "H": 2048, "F": 768, "skew": 0.5},
        {"name": "experts_down_t4096", "op": "down", "T": 4096, "E": 128, "k": 8, "H": 2048, "F": 768, "skew": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        if rng.random() < 0.5:
            c = {"op": "lora", "T": _log_int(rng, 1, 4096), "N": 8 * _log_int(rng, 16, 1728), "K": 8 * _log_int(rng, 16, 1728),
                 "r": 8 * rng.randint(1, 16), "n": _log_int(rng, 1, 64), "epi": rng.choice(["store", "gelu", "resid", "swiglu"])}
            c["reqs"] = min(c["T"], _log_int(rng, 1, 64))
            two = 2 if c["epi"] == "swiglu" else 1
            if two * c["N"] * c["K"] <= 2 * 13824 * 5120 and two * c["T"] * c["N"] * c["K"] <= 2 * 2048 * 13824 * 5120:
                return c
        else:
            c = {"op": rng.choice(["up", "down"]), "T": _log_int(rng, 1, 4096), "E": rng.randint(8, 256), "k": rng.randint(1, 8),
                 "H": 8 * _log_int(rng, 32, 512), "F": 8 * _log_int(rng, 16, 256), "skew": rng.choice([0.0, 0.5, 1.0, 2.0])}
            if (c["E"] * c["H"] * c["F"] <= 128 * 2048 * 768
                    and c["T"] * c["k"] * c["H"] * c["F"] <= 4096 * 8 * 2048 * 768):
                return c


# ------------------------------------------------------------------ inputs
def _normal(g, shape, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _pitches(K):
    return -(-K // 128) * 64, -(-K // 512) * 16


def _pack(v):
    """MXFP4 codes and scales of [E, rows, K] values."""
    pad = -v.shape[-1] % 128
    v = torch.nn.functional.pad(v, (0, pad)) if pad else v
    v = v.reshape(*v.shape[:-1], -1, 32)
    amax = v.abs().amax(-1)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    s = s.clamp(-127, 125)
    a = (v * ((127 - s) << 23).view(torch.float32)[..., None]).abs()   # times 2^-s, exactly
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = mag + 8 * (v < 0).to(torch.uint8)
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, -s.shape[-1] % 16))
    return byte.flatten(-2).contiguous(), scales.contiguous()


def _pack_experts(g, E, rows, K):
    cp, sp = _pitches(K)
    codes = torch.empty((E, rows, cp), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, rows, sp), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (rows * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n], scales[e:e + n] = _pack(_normal(g, (n, rows, K), K ** -0.5))
    return codes, scales


def _requests(g, case):
    """The adapter of each row: requests' rows lie together; about one request in eight has none."""
    T, q = case["T"], case["reqs"]
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:q - 1].add_(1).sort().values if q > 1 else torch.empty(0, device="cuda", dtype=torch.int64)
    of = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    each = torch.randint(0, case["n"], (q,), generator=g, device="cuda")
    each = torch.where(torch.rand(q, generator=g, device="cuda") < 0.125, -1, each)
    return each[of].to(torch.int32)


def _routing(g, case):
    """What the routing of a layer leaves: row table, group bounds and weights."""
    T, E = case["T"], case["E"]
    k = min(case["k"], E)
    logits = _normal(g, (T, E)) + case["skew"] * _normal(g, (1, E))
    top, sel = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, sel = top[:, :k], sel[:, :k].reshape(-1)
    table = torch.sort(sel, stable=True).indices.to(torch.int32)
    bounds = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    bounds[1:] = torch.bincount(sel, minlength=E).cumsum(0)
    ex = torch.exp(top - top[:, :1])
    return k, table, bounds, (ex / ex.sum(-1, keepdim=True)).reshape(-1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2 + 1)
    st = {"case": case}
    if case["op"] == "lora":
        T, N, K, r, n = (case[i] for i in ("T", "N", "K", "r", "n"))
        two = 2 if case["epi"] == "swiglu" else 1
        st["x"] = _normal(g, (T, K), dtype=torch.bfloat16)
        st["w"] = _normal(g, (two * N, K), K ** -0.5, torch.bfloat16)
        st["down"] = _normal(g, (n, two * r, K), K ** -0.5, torch.bfloat16)
        st["up"] = _normal(g, (n, N, r), r ** -0.5, torch.bfloat16)
        st["up2"] = _normal(g, (n, N, r), r ** -0.5, torch.bfloat16) if two == 2 else None
        st["scale"] = 0.25 + torch.rand(n, generator=g, device="cuda")
        st["ids"] = _requests(g, case)
        if case["epi"] in ("gelu", "resid"):
            st["bias"] = _normal(g, (N,), 0.5, torch.bfloat16)
        if case["epi"] == "resid":
            st["resid"] = _normal(g, (T, N))
        if own:
            from host_offloaded_weight_gb300 import lstream as L
            st["lora"] = L.lsk_lora_adapters(st["down"], st["up"], up2=st["up2"], scale=st["scale"])
        return st
    E, H, F = case["E"], case["H"], case["F"]
    st["k"], st["table"], st["bounds"], st["weight"] = _routing(g, case)
    st["bounds_host"] = st["bounds"].tolist()
    if case["op"] == "up":
        st["x"] = _normal(g, (case["T"], H), dtype=torch.bfloat16)
        st["gate"], st["gate_scales"] = _pack_experts(g, E, F, H)
        st["up"], st["up_scales"] = _pack_experts(g, E, F, H)
    else:
        # a hidden activation: the product of two normal values, most of them small
        h = _normal(g, (case["T"] * st["k"], F))
        st["h"] = (h * torch.sigmoid(h) * _normal(g, h.shape)).to(torch.bfloat16)
        st["down"], st["down_scales"] = _pack_experts(g, E, H, F)
    return st


# ------------------------------------------------------------------ the framework's operators
def _run_own(st):
    from host_offloaded_weight_gb300 import lstream as L
    case = st["case"]
    if case["op"] == "lora":
        T, N, K, epi = case["T"], case["N"], case["K"], case["epi"]
        out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        if epi == "store":
            L.lsk_gemm_lora_bf16(L.LSK_EPI_STORE, st["x"], st["w"], st["lora"], st["ids"], out, T, N, K)
        elif epi == "gelu":
            L.lsk_gemm_lora_bf16(L.LSK_EPI_BIAS_GELU, st["x"], st["w"], st["lora"], st["ids"], out, T, N, K, bias=st["bias"])
        elif epi == "swiglu":
            L.lsk_gemm_lora_bf16(L.LSK_EPI_SWIGLU, st["x"], st["w"], st["lora"], st["ids"], out, T, N, K, b2_row_off=N)
        else:
            out32 = torch.empty((T, N), dtype=torch.float32, device="cuda")
            L.lsk_gemm_lora_bf16(L.LSK_EPI_BIAS_RESID, st["x"], st["w"], st["lora"], st["ids"], out, T, N, K, bias=st["bias"],
                                 resid=st["resid"], C32=out32)
            return out, out32
        return out
    E, H, F, M = case["E"], case["H"], case["F"], case["T"] * st["k"]
    if case["op"] == "up":
        out = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
        L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SWIGLU, st["x"], st["gate"], st["gate_scales"], st["bounds"], E, out, M, F, H,
                                      B2_codes=st["up"], B2_scales=st["up_scales"], row_table=st["table"], gather_k=st["k"])
        return out
    out = torch.empty((M, H), dtype=torch.float32, device="cuda")
    L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SCALE_F32, st["h"], st["down"], st["down_scales"], st["bounds"], E, out, M, H, F,
                                  row_table=st["table"], row_weight=st["weight"])
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
    if case["op"] == "lora":
        N, r, epi = case["N"], case["r"], case["epi"]
        x = st["x"].float()
        z = x @ st["w"].float().T
        for a in range(case["n"]):
            on = ((st["ids"] == a).float() * st["scale"][a])[:, None]
            h = (x @ st["down"][a].float().T) * on
            z[:, :N] += h[:, :r] @ st["up"][a].float().T
            if epi == "swiglu":
                z[:, N:] += h[:, r:] @ st["up2"][a].float().T
        if epi == "store":
            return z.to(torch.bfloat16)
        if epi == "swiglu":
            return (z[:, :N] / (1.0 + torch.exp(-z[:, :N])) * z[:, N:]).to(torch.bfloat16)
        z += st["bias"].float()
        if epi == "gelu":
            return (0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))).to(torch.bfloat16)
        z += st["resid"]
        return z.to(torch.bfloat16), z
    E, H, F, M = case["E"], case["H"], case["F"], case["T"] * st["k"]
    at = st["bounds_host"]
    table = st["table"].long()
    if case["op"] == "up":
        rows = st["x"].float()[table // st["k"]]
        out = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            if at[e] == at[e + 1]:
                continue
            a = rows[at[e]:at[e + 1]] @ _decode(st["gate"][e], st["gate_scales"][e], H).T
            b = rows[at[e]:at[e + 1]] @ _decode(st["up"][e], st["up_scales"][e], H).T
            out[at[e]:at[e + 1]] = (a / (1.0 + torch.exp(-a)) * b).to(torch.bfloat16)
        return out
    rows = st["h"].float()
    y = torch.empty((M, H), dtype=torch.float32, device="cuda")
    for e in range(E):
        if at[e] < at[e + 1]:
            y[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ _decode(st["down"][e], st["down_scales"][e], F).T
    out = torch.empty_like(y)
    out[table] = y * st["weight"][table][:, None]
    return out


# ------------------------------------------------------------------ 64 bits
def _exact_matrix(codes, scales, K):
    """Values from the format's bit fields: sign, two exponent bits (bias 1), one mantissa bit."""
    c = torch.stack((codes % 16, torch.div(codes, 16, rounding_mode="floor")), -1).flatten(-2)[..., :K].to(torch.int64)
    sign, e, m = 1.0 - 2.0 * (c // 8).double(), (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    unit = ((scales.to(torch.int64) - 127 + 1023) << 52).view(torch.float64)   # 2^(byte - 127), exactly
    return sign * mag * unit[..., torch.arange(K, device=codes.device) // 32]


def exact(case, seed):
    if work(case)["flops"] > 1e12:   # the 64-bit products of more would take long
        return None
    st = prepare(case, seed)
    if case["op"] == "lora":
        T, N, K, r, epi = (case[i] for i in ("T", "N", "K", "r", "epi"))
        ids = st["ids"].tolist()
        used = sorted({a for a in ids if a >= 0})
        x = st["x"].double()
        h = torch.zeros((T, st["down"].shape[1]), dtype=torch.float64, device="cuda")
        rows = {a: torch.tensor([t for t in range(T) if ids[t] == a], device="cuda") for a in used}
        for a in used:
            h[rows[a]] = float(st["scale"][a]) * (x[rows[a]] @ st["down"][a].double().T)

        def product(w, up, h):
            z = torch.cat([x @ p.double().T for p in w.split(1024)], 1)
            for a in used:
                z[rows[a]] += h[rows[a]] @ up[a].double().T
            return z

        z = product(st["w"][:N], st["up"], h[:, :r])
        if epi == "store":
            return z
        if epi == "swiglu":
            return z * torch.sigmoid(z) * product(st["w"][N:], st["up2"], h[:, r:])
        z = z + st["bias"].double()
        if epi == "gelu":
            return z * torch.special.ndtr(z)
        z = z + st["resid"].double()
        return z, z
    H, F, k = case["H"], case["F"], st["k"]
    table, at = st["table"].tolist(), st["bounds_host"]
    if case["op"] == "up":
        out = torch.zeros((len(table), F), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            if at[e + 1] > at[e]:
                x = st["x"][[i // k for i in table[at[e]:at[e + 1]]]].double()
                a = x @ _exact_matrix(st["gate"][e], st["gate_scales"][e], H).T
                out[at[e]:at[e + 1]] = a * torch.sigmoid(a) * (x @ _exact_matrix(st["up"][e], st["up_scales"][e], H).T)
        return out
    out = torch.zeros((len(table), H), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            to = table[at[e]:at[e + 1]]
            y = st["h"][at[e]:at[e + 1]].double() @ _exact_matrix(st["down"][e], st["down_scales"][e], F).T
            out[to] = y * st["weight"][to].double()[:, None]
    return out


# ------------------------------------------------------------------ least work
def work(case):
    if case["op"] == "lora":
        T, N, K, r = case["T"], case["N"], case["K"], case["r"]
        two = 2 if case["epi"] == "swiglu" else 1
        used = case["n"] * (1 - (1 - 0.875 / case["n"]) ** case["reqs"])   # expected number of adapters with a row
        values = T * K + two * N * K + T * N + two * used * r * (N + K)
        more = {"store": 0, "gelu": 2 * N, "swiglu": 0, "resid": 2 * N + 8 * T * N}[case["epi"]]
        return {"bytes": 2 * values + more + 4 * T, "flops": 2 * two * T * N * K + 2 * two * 0.875 * T * r * (N + K)}
    T, E, H, F = case["T"], case["E"], case["H"], case["F"]
    k = min(case["k"], E)
    used = E * (1 - (1 - k / E) ** T)   # expected number of experts with a row (an even routing's)
    if case["op"] == "up":
        return {"bytes": used * 2 * H * F * 17 / 32 + 2 * T * H + 2 * T * k * F + 4 * T * k, "flops": 4 * T * k * H * F}
    return {"bytes": used * H * F * 17 / 32 + 2 * T * k * F + 4 * T * k * H + 8 * T * k, "flops": 2 * T * k * H * F}
