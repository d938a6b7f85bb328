"""A mixture-of-experts perceptron trained and then served with this library's products.

    python examples/moe_layer.py

Each token goes to the two experts that a router picks; expert e computes GELU(x W1_e + b1_e) W2_e +
b2_e.  The rows are sorted by expert on the device, and the offsets of the groups never reach the host.

  training   run_grouped        forward, and (with the weights' other layout) the data gradient
             run_grouped_wgrad  weight and bias gradients; with alpha = -rate and beta = 1 the call
                                is the update of the weights itself
  serving    quantize_rows      the weights once (a scale for each output channel), the activations
                                of each call (a scale for each token)
             run_grouped_i8     the same layer in 8-bit integers, bias and GELU in the epilogue
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import tiled_matrix_multiply_amd as tmm

BIAS, GELU = tmm.GEMM_EPI_BIAS, tmm.GEMM_EPI_GELU


def sort_by_expert(scores, experts, top=2):
    """Rows of the sorted batch: the token of each, its weight, and the groups' offsets (int64)."""
    weight, expert = scores.topk(top, dim=1)
    order = expert.flatten().argsort(stable=True)
    sorted_expert = expert.flatten()[order]
    offsets = torch.searchsorted(sorted_expert, torch.arange(experts + 1, device=scores.device))
    return order // top, torch.softmax(weight, dim=1).flatten()[order], offsets


class Layer:
    """Two grouped products; weights are stored N x K (a row for each output channel)."""

    def __init__(self, handle, experts, dim, hidden, gen):
        def normal(*shape, scale):
            return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(torch.bfloat16)

        self.h, self.experts, self.dim, self.hidden = handle, experts, dim, hidden
        self.w1 = normal(experts, hidden, dim, scale=dim ** -0.5)
        self.w2 = normal(experts, dim, hidden, scale=hidden ** -0.5)
        self.b1 = torch.zeros(experts, hidden, device="cuda")
        self.b2 = torch.zeros(experts, dim, device="cuda")

    def product(self, x, w, bias, offsets, epilogue):
        rows, k = x.shape
        y = torch.empty(rows, w.shape[1], device="cuda", dtype=x.dtype)
        self.h.run_grouped(x, w, y, offsets, groups=self.experts, M=rows, N=w.shape[1], K=k,
                           trans_b=True, epilogue=epilogue, bias=bias)
        return y

    def forward(self, x, offsets):
        h = self.product(x, self.w1, self.b1, offsets, BIAS | GELU)
        return self.product(h, self.w2, self.b2, offsets, BIAS)

    def data_grad(self, dy, w, offsets):
        rows, k = dy.shape
        dx = torch.empty(rows, w.shape[2], device="cuda", dtype=dy.dtype)
        self.h.run_grouped(dy, w, dx, offsets, groups=self.experts, M=rows, N=w.shape[2], K=k,
                           trans_b=False)
        return dx

    def update(self, x, dy, w, b, offsets, rate):
        """w -= rate * the weight gradient, in place; b likewise."""
        db = torch.empty_like(b)
        self.h.run_grouped_wgrad(x, dy, w, offsets, groups=self.experts, M=x.shape[0], N=w.shape[1],
                                 K=w.shape[2], trans_b=True, alpha=-rate, beta=1.0, dbias=db)
        b -= rate * db

    def train_step(self, x, target, offsets, rate):
        z = self.product(x, self.w1, self.b1, offsets, BIAS)
        h = torch.nn.functional.gelu(z.float()).to(z.dtype)
        y = self.product(h, self.w2, self.b2, offsets, BIAS)
        error = y.float() - target
        dy = error.to(y.dtype)
        dh = self.data_grad(dy, self.w2, offsets).float()
        zf = z.float()
        slope = 0.5 * torch.erfc(zf * -(0.5 ** 0.5)) + zf * torch.exp(-0.5 * zf * zf) * (2 * torch.pi) ** -0.5
        self.update(h, dy, self.w2, self.b2, offsets, rate)
        self.update(x, (dh * slope).to(z.dtype), self.w1, self.b1, offsets, rate)
        return 0.5 * (error * error).sum() / x.shape[0]


class Layer8:
    """The trained layer in 8-bit integers."""

    def __init__(self, layer):
        self.h, self.experts = layer.h, layer.experts
        self.b1, self.b2 = layer.b1, layer.b2
        self.w1, self.s1 = self.codes(layer.w1)
        self.w2, self.s2 = self.codes(layer.w2)

    def codes(self, x):
        """8-bit integers of the rows of x and a scale for each row."""
        k = x.shape[-1]
        rows = x.numel() // k
        q = torch.empty(x.shape, device="cuda", dtype=torch.int8)
        s = torch.empty(x.shape[:-1], device="cuda")
        self.h.quantize_rows(x, q, s, M=rows, K=k)
        return q, s

    def product(self, x, w, sw, bias, offsets, epilogue):
        q, s = self.codes(x)
        y = torch.empty(x.shape[0], w.shape[1], device="cuda", dtype=x.dtype)
        self.h.run_grouped_i8(q, s, w, sw, y, offsets, groups=self.experts, M=x.shape[0],
                              N=w.shape[1], K=x.shape[1], trans_b=True, epilogue=epilogue, bias=bias)
        return y

    def forward(self, x, offsets):
        h = self.product(x, self.w1, self.s1, self.b1, offsets, BIAS | GELU)
        return self.product(h, self.w2, self.s2, self.b2, offsets, BIAS)


def main(tokens=512, dim=256, hidden=768, experts=8, steps=40, rate=1e-4, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    with tmm.Gemm(0) as handle:
        layer = Layer(handle, experts, dim, hidden, gen)
        x = torch.randn(tokens, dim, device="cuda", generator=gen).to(torch.bfloat16)
        scores = torch.randn(tokens, experts, device="cuda", generator=gen)
        token, weight, offsets = sort_by_expert(scores, experts)
        rows = x[token]
        target = torch.randn(tokens, dim, device="cuda", generator=gen)[token]
        losses = [layer.train_step(rows, target, offsets, rate) for _ in range(steps)]

        def combine(y):  # the experts' answers for each token, by the router's weights
            return torch.zeros(tokens, dim, device="cuda").index_add_(0, token, y.float() * weight[:, None])

        y16 = combine(layer.forward(rows, offsets))
        y8 = combine(Layer8(layer).forward(rows, offsets))
        off = ((y8 - y16).norm() / y16.norm()).item()
        losses = [l.item() for l in losses]
        print(f"loss a row: {losses[0]:.2f} -> {losses[-1]:.2f} in {steps} steps; "
              f"8-bit output within {100 * off:.2f}% of the bf16 one")
        return losses, off


if __name__ == "__main__":
    main()
