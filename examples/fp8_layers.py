"""8-bit layers from the library's calls: a linear layer trained for some steps, and
a mixture-of-experts layer decoding a few tokens.

    python examples/fp8_layers.py [--steps 20] [--tokens 512] [--width 512]

Training: y = x W^T.  Activations and gradients are quantised with one scale for
each 128 along the dimension that the product sums over, weights with one for
each 128 x 128 block:

    forward    y  = x W^T    x 1 x 128,   W blocks,    layout NT
    input      dx = dy W     dy 1 x 128,  W blocks,    layout NN (W's codes as they are)
    weights    dW += dy^T x  dy, x 128 x 1 (along the tokens), layout TN, fp32, beta = 1

Decoding: the experts' matrices are quantised once, in blocks, into rows that start
on 16 bytes; each step is one call for the whole layer.

Needs a GB300 and the built library.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import dense_fp32_gemm_05_gb300 as sg  # noqa: E402

BLOCKS = (128, 128)


class Linear8:
    """y = x W^T with fp32 master weights."""

    def __init__(self, n, k, device, generator):
        self.w = torch.randn((n, k), device=device, generator=generator) / k ** 0.5
        self.dw = torch.zeros_like(self.w)
        self.quantize()

    def quantize(self):
        self.qw, self.sw = sg.fp8_quantize(self.w, BLOCKS)

    def forward(self, x):
        self.x = x
        qx, sx = sg.fp8_quantize(x)
        y = torch.empty((x.shape[0], self.w.shape[0]), device=x.device, dtype=torch.bfloat16)
        return sg.fp8_gemm(qx, sx, self.qw, self.sw, y)

    def backward(self, dy):
        """dx, and dW added to self.dw; gradients in E5M2 (their range is wider)."""
        qdy, sdy = sg.fp8_quantize(dy, (1, 128), torch.float8_e5m2)
        dx = sg.fp8_gemm(qdy, sdy, self.qw, self.sw, torch.empty_like(self.x), "N", "N")
        qt, st = sg.fp8_quantize(dy, (128, 1), torch.float8_e5m2)
        xt, sx = sg.fp8_quantize(self.x, (128, 1))
        sg.fp8_gemm(qt, st, xt, sx, self.dw, "T", "N", beta=1.0, b_group=1)
        return dx

    def step(self, rate):
        self.w.sub_(self.dw, alpha=rate)
        self.dw.zero_()
        self.quantize()


def train(steps, tokens, width, device="cuda"):
    """Fits a linear map by gradient descent; returns the losses."""
    g = torch.Generator(device=device).manual_seed(0)
    target = torch.randn((width, width), device=device, generator=g) / width ** 0.5
    layer = Linear8(width, width, device, g)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, width), device=device, generator=g).to(torch.bfloat16)
        want = x.float() @ target.t()
        error = layer.forward(x).float() - want
        losses.append(float(error.square().mean()))
        layer.backward((error * (2.0 / tokens)).to(torch.bfloat16))
        layer.step(0.1)
    return losses


class Experts8:
    """Quantised gate, up and down matrices of every expert, and the router."""

    def __init__(self, experts, width, inner, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.router = torch.randn((experts, width), device=device, generator=g) / width ** 0.5
        self.codes, self.scales = {}, {}
        for name, n, k in (("gate", inner, width), ("up", inner, width), ("down", width, inner)):
            ld = (k + 15) // 16 * 16
            codes = torch.empty((experts, n, ld), device=device, dtype=torch.float8_e4m3fn)[:, :, :k]
            scales = torch.empty((experts, (n + 127) // 128, (k + 127) // 128), device=device)
            for e in range(experts):
                w = torch.randn((n, k), device=device, generator=g) / k ** 0.5
                sg.fp8_quantize(w, BLOCKS, Q=codes[e], S=scales[e])
            self.codes[name], self.scales[name] = codes, scales

    def __call__(self, x, topk, **buffers):
        c, s = self.codes, self.scales
        return sg.moe(x, self.router, c["gate"], s["gate"], c["up"], s["up"], c["down"], s["down"], topk,
                      **buffers)


def decode(tokens, steps, experts=16, width=1024, inner=512, topk=4, device="cuda"):
    """Feeds the layer's output back to it (residual, normalised) for some steps."""
    layer = Experts8(experts, width, inner, device)
    x = torch.randn((tokens, width), device=device, generator=torch.Generator(device=device).manual_seed(1))
    x = x.to(torch.bfloat16)
    for _ in range(steps):
        y, _, indices, _ = layer(x, topk)
        x = torch.nn.functional.layer_norm((x + y).float(), (width,)).to(torch.bfloat16)
    return x, indices


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=512)
    a = ap.parse_args()
    losses = train(a.steps, a.tokens, a.width)
    print("training loss: " + " ".join(f"{v:.4f}" for v in losses))
    x, indices = decode(4, a.steps)
    print(f"decoded {a.steps} steps of 4 tokens; the last step's experts: {indices.tolist()}")
    status = sg.sgemm_device_error(torch.cuda.current_stream())
    print("device error word:", sg.sgemm_status_string(status))
    return 0 if status == sg.SGEMM_OK and losses[-1] < 0.1 * losses[0] else 1


if __name__ == "__main__":
    sys.exit(main())
