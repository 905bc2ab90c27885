"""Decode steps of a stack of MoE layers whose MXFP4 experts stream from pinned host memory.

Each layer is y = x + sum_j w_j D_e(SiLU(G_e x) * (U_e x)) with a router of its own, and a head
gives the logits of the vocabulary at the end. All matrices are quantised once on the device
(lsk_mxfp4_quantize) and kept in pinned host memory, one blob a layer: a bf16 layer takes 3.74
times its bytes of the host link (default sizes). A step runs, per layer, the copy of a later layer's blob into
the slot that has become free (copy stream) beside the router's product (lsk_gemm_bf16_mxfp4,
fp32 logits) and the experts (lsk_moe_few) out of the active slot. The head stays on the device:
a few tokens go through lsk_gemm_bf16_mxfp4, a prompt's many rows through lsk_gemm_mxfp4 with the
activations quantised on the way.

    python examples/mxfp4_moe_decode.py --layers 16 --experts 64 --hidden 2048 --ffn 768 --tokens 8
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from host_offloaded_weight_gb300 import lstream as L  # noqa: E402

COPY_CTAS = 24       # enough for the host link's rate; the other SMs stay free of copies
FEW = 64             # tokens up to which the products keep bf16 activations


def mx_matrix(rows, K):
    """Codes and scales of a [rows, K] matrix (uninitialised, on the device)."""
    return (torch.empty((rows, L.lsk_mxfp4_code_pitch(K)), dtype=torch.uint8, device="cuda"),
            torch.empty((rows, L.lsk_mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda"))


def quantise(w):
    """[rows, K] bf16 or fp32 on the device -> (codes, scales)."""
    codes, scales = mx_matrix(*w.shape)
    L.lsk_mxfp4_quantize(w, w.shape[0], w.shape[1], codes, scales)
    return codes, scales


class Layout:
    """Where a layer's matrices lie in its blob (offsets of whole 256-byte units)."""

    def __init__(self, E, H, F):
        self.E, self.H, self.F = E, H, F
        self.at, self.nbytes = {}, 0
        for name, rows, K in (("router", E, H), ("gate", E * F, H), ("up", E * F, H), ("down", E * H, F)):
            for part, pitch in (("codes", L.lsk_mxfp4_code_pitch(K)), ("scales", L.lsk_mxfp4_scale_pitch(K))):
                self.at[name, part] = (self.nbytes, rows, pitch)
                self.nbytes += -(-rows * pitch // 256) * 256

    def view(self, blob, name, part, per=None):
        o, rows, pitch = self.at[name, part]
        t = blob[o:o + rows * pitch].view(rows, pitch)
        return t if per is None else t.view(self.E, per, pitch)


class Stack:
    """Layers in pinned host memory, two slots on the device, and the head."""

    def __init__(self, layers, E, H, F, vocab, k, seed=0):
        self.n, self.k, self.vocab = layers, k, vocab
        self.lay = Layout(E, H, F)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def random(rows, K):
            return quantise((torch.randn((rows, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16))

        self.host = []
        for _ in range(layers):
            blob = torch.zeros(self.lay.nbytes, dtype=torch.uint8).pin_memory()
            for name, rows, K in (("router", E, H), ("gate", E * F, H), ("up", E * F, H), ("down", E * H, F)):
                for part, t in zip(("codes", "scales"), random(rows, K)):
                    self.lay.view(blob, name, part).copy_(t)
            self.host.append(blob)
        self.head = random(vocab, H)
        self.slots = torch.empty((2, self.lay.nbytes), dtype=torch.uint8, device="cuda")
        self.ready = torch.zeros(2, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32).pin_memory()
        self.copies, self.compute = torch.cuda.Stream(), torch.cuda.Stream()
        self.free = [torch.cuda.Event() for _ in range(2)]
        self.loads = 0
        torch.cuda.synchronize()

    def load(self, layer):
        """Queues the layer's copy into the next slot, after the work that still reads that slot."""
        s = self.loads % 2
        self.copies.wait_event(self.free[s])
        self.loads += 1
        L.lsk_copy_h2slot_static(self.slots[s], [self.host[layer]], [self.lay.nbytes], [0], COPY_CTAS,
                                 self.ready[s:], self.loads, stream=self.copies)
        return s, self.loads

    def layer(self, blob, x, out, logits):
        """One layer out of a blob on the device, on the compute stream."""
        E, H, F, T = self.lay.E, self.lay.H, self.lay.F, x.shape[0]
        v = self.lay.view
        L.lsk_gemm_bf16_mxfp4(x, v(blob, "router", "codes"), v(blob, "router", "scales"), logits, T, E, H,
                              stream=self.compute)
        L.lsk_moe_few(x, logits, v(blob, "gate", "codes", F), v(blob, "up", "codes", F), v(blob, "down", "codes", H),
                      T, E, self.k, H, F, out, gate_scales=v(blob, "gate", "scales", F),
                      up_scales=v(blob, "up", "scales", F), down_scales=v(blob, "down", "scales", H),
                      stream=self.compute)

    def logits(self, x):
        """The head's product for the rows of x, fp32; ordered with the caller's stream on both sides."""
        M, H = x.shape
        self.compute.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.compute):
            out = torch.empty((M, self.vocab), dtype=torch.float32, device="cuda")
            if M <= FEW:
                L.lsk_gemm_bf16_mxfp4(x, *self.head, out, M, self.vocab, H)
            else:
                L.lsk_gemm_mxfp4(*quantise(x), *self.head, out, M, self.vocab, H)
        torch.cuda.current_stream().wait_stream(self.compute)
        return out

    def step(self, x):
        """x [T, H] bf16, T <= 64 -> the head's logits [T, vocab], layers streamed."""
        self.compute.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.compute):
            bufs = [x, torch.empty_like(x), torch.empty_like(x)]
            logits = torch.empty((x.shape[0], self.lay.E), dtype=torch.float32, device="cuda")
        queued = [self.load(i) for i in range(min(2, self.n))]
        for i in range(self.n):
            s, epoch = queued[i]
            L.lsk_wait_ready(self.ready[s:], epoch, 2000, self.err, s, stream=self.compute)
            self.layer(self.slots[s], bufs[0 if i == 0 else 1 + (i - 1) % 2], bufs[1 + i % 2], logits)
            self.free[s].record(self.compute)
            if i + 2 < self.n:
                queued.append(self.load(i + 2))
        return self.logits(bufs[1 + (self.n - 1) % 2])

    def check(self):
        """After a synchronise: raises if a copy did not arrive or a kernel's wait ran out."""
        err = int(self.err[0]) or L.lsk_device_error()
        if err:
            raise RuntimeError(f"device error word {err:#x}")


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("layers", 16), ("experts", 64), ("hidden", 2048), ("ffn", 768), ("vocab", 32000),
                          ("top-k", 8), ("tokens", 8), ("prompt", 1024), ("steps", 10)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    st = Stack(a.layers, a.experts, a.hidden, a.ffn, a.vocab, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    prompt = torch.randn((a.prompt, a.hidden), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    for _ in range(3):
        out = st.step(x)
    scores = st.logits(prompt)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        out = st.step(x)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / a.steps
    st.check()
    nbytes = a.layers * st.lay.nbytes
    bf16 = a.layers * 2 * a.hidden * a.experts * (3 * a.ffn + 1)
    print(f"{a.tokens} tokens a step: {dt * 1e3:.2f} ms, {a.tokens / dt:.0f} tokens/s; {nbytes / 1e6:.0f} MB of MXFP4 a step "
          f"at {nbytes / dt / 1e9:.0f} GB/s (bf16 would be {bf16 / 1e6:.0f} MB)")
    print(f"next tokens {out.argmax(1).tolist()[:8]}; prompt scores {tuple(scores.shape)}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
