"""A layer of a prompt of several requests, from the library's own calls: the shared projection with each request's adapter, routing, and
MXFP4 experts grouped by ragged sizes; once by itself, once captured and replayed on other inputs, and some layers in a row."""
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Layer:
    def __init__(self, H, F, E, k, r, n, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.H, self.F, self.E, self.k, self.n = H, F, E, k, n
        self.w = normal(H, H, scale=H ** -0.5).to(BF16)
        self.down = normal(n, r, H, scale=H ** -0.5).to(BF16)
        self.up = normal(n, H, r, scale=r ** -0.5).to(BF16)
        self.scale = 0.5 + torch.rand(n, generator=g, device="cuda")
        self.lora = L.lsk_lora_adapters(self.down, self.up, scale=self.scale)
        self.mats = {}
        for name, rows, K in (("gate", F, H), ("up", F, H), ("down", H, F)):
            v = normal(E * rows, K, scale=K ** -0.5)
            c = torch.empty((E, rows, L.lsk_mxfp4_code_pitch(K)), dtype=torch.uint8, device="cuda")
            s = torch.empty((E, rows, L.lsk_mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda")
            L.lsk_mxfp4_quantize(v, E * rows, K, c, s)
            back = torch.empty((E * rows, K), device="cuda")
            L.lsk_mxfp4_dequantize(c, s, E * rows, K, back)
            self.mats[name] = c, s, back.double().unflatten(0, (E, rows))

    def buffers(self, T):
        H, F, E, k = self.H, self.F, self.E, self.k
        i32 = {"dtype": torch.int32, "device": "cuda"}
        return {"y": torch.empty((T, H), dtype=BF16, device="cuda"), "y32": torch.empty((T, H), device="cuda"), "sel": torch.empty((T, k), **i32),
                "weight": torch.empty((T, k), device="cuda"), "table": torch.empty(T * k, **i32), "bounds": torch.empty(E + 1, **i32),
                "h": torch.empty((T * k, F), dtype=BF16, device="cuda"), "z": torch.empty((T * k, H), device="cuda"),
                "out": torch.empty((T, H), dtype=BF16, device="cuda"), "out32": torch.empty((T, H), device="cuda")}

    def run(self, x, x32, ids, logits, b):
        T, H, F, E, k = x.shape[0], self.H, self.F, self.E, self.k
        m = self.mats
        L.lsk_gemm_lora_bf16(L.LSK_EPI_RESID, x, self.w, self.lora, ids, b["y"], T, H, H, resid=x32, C32=b["y32"])
        L.lsk_moe_route(logits, 1, T, E, k, b["sel"], b["weight"])
        L.lsk_moe_group(b["sel"], 1, T, E, k, b["table"], b["bounds"])
        L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SWIGLU, b["y"], *m["gate"][:2], b["bounds"], E, b["h"], T * k, F, H, B2_codes=m["up"][0],
                                      B2_scales=m["up"][1], row_table=b["table"], gather_k=k)
        L.lsk_gemm_grouped_bf16_mxfp4(L.LSK_EPI_SCALE_F32, b["h"], *m["down"][:2], b["bounds"], E, b["z"], T * k, H, F, row_table=b["table"],
                                      row_weight=b["weight"])
        L.lsk_moe_combine(b["y32"], b["z"], T, k, H, b["out"], b["out32"])

    def check(self, x, x32, ids, b):
        torch.cuda.synchronize()
        assert L.lsk_device_error() == 0
        want, size = x.double() @ self.w.double().T, x.double().abs() @ self.w.double().abs().T
        for a in range(self.n):
            rows = torch.nonzero(ids == a).flatten()
            if len(rows):
                s, d, u = float(self.scale[a]), self.down[a].double(), self.up[a].double()
                want[rows] += s * (x[rows].double() @ d.T) @ u.T
                size[rows] += s * (x[rows].double().abs() @ d.abs().T) @ u.abs().T
        want += x32.double()
        # sums of H products and of the adapter's in fp32, three terms of h (24 bits)
        tol = (self.H + 64) * 2.0 ** -23 * size + 2.0 ** -22 * want.abs()
        assert bool(((b["y32"].double() - want).abs() <= tol).all())
        assert bool(((b["y"].double() - b["y32"].double()).abs() <= 2.0 ** -8 * b["y32"].double().abs()).all())
        # the experts, from the projection's own rounded result
        y, out, size = b["y"].double(), b["y32"].double(), b["y32"].double().abs()
        for e in range(self.E):
            rows, j = torch.nonzero(b["sel"] == e, as_tuple=True)
            if not len(rows):
                continue
            g, u, d = (self.mats[n][2][e] for n in ("gate", "up", "down"))
            a = y[rows] @ g.T
            hid, w = a * torch.sigmoid(a) * (y[rows] @ u.T), b["weight"][rows, j].double()[:, None]
            out.index_add_(0, rows, w * (hid @ d.T))
            size.index_add_(0, rows, w * (hid.abs() @ d.abs().T))
        # the hidden activation's rounding to bf16, half a step of each value; the fp32 sums are far below it
        assert bool(((b["out32"].double() - out).abs() <= (2.0 ** -8 + 2.0 ** -12) * size).all())


def _inputs(T, layer, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x32 = torch.randn((T, layer.H), generator=g, device="cuda")
    x = x32.to(BF16)
    each = torch.randint(-1, layer.n, (5,), generator=g, device="cuda").to(torch.int32)     # five requests
    ids = each[torch.arange(T, device="cuda") * 5 // max(T, 1)]
    return x, x32, ids.contiguous(), torch.randn((T, layer.E), generator=g, device="cuda")


@pytest.mark.parametrize("T", [1, 7, 64, 65, 150, 700])
def test_a_prompt_through_a_layer(T):
    layer = Layer(264, 136, 12, 3, 16, 6, seed=T)
    x, x32, ids, logits = _inputs(T, layer, T)
    b = layer.buffers(T)
    layer.run(x, x32, ids, logits, b)
    layer.check(x, x32, ids, b)


@pytest.mark.parametrize("T", [20, 300])
def test_captured_and_replayed_on_other_prompts(T):
    layer = Layer(256, 128, 16, 4, 24, 5, seed=3)
    bufs, ins = layer.buffers(T), _inputs(T, layer, 1)
    layer.run(*ins, bufs)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        layer.run(*ins, bufs)
    for seed in (2, 3, 4):
        for t, new in zip(ins, _inputs(T, layer, seed)):
            t.copy_(new)
        g.replay()
        layer.check(ins[0], ins[1], ins[2], bufs)


def test_layers_in_a_row_have_the_bits_of_layers_one_by_one():
    layers = [Layer(256, 192, 8, 2, 16, 4, seed=i) for i in range(4)]
    results = []
    for wait in (True, False, False):
        x, x32, ids, logits = _inputs(200, layers[0], 9)
        for layer in layers:
            b = layer.buffers(200)
            layer.run(x, x32, ids, logits, b)
            x, x32 = b["out"], b["out32"]
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(x32.clone())
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
