"""A mixture-of-experts perceptron trained and then served with this library's products.

    python examples/moe_layer.py

Each token goes to the two experts that a router picks; expert e computes GELU(x W1_e + b1_e) W2_e +
b2_e.  The rows are sorted by expert on the device, and the offsets of the groups never reach the host.

  routing    route              the experts of each token, their weights, the rows' order and the offsets
             dispatch_rows      the tokens' rows into that order
             combine_rows       each token's answers back, by the router's weights
  training   run_grouped        forward, and (with the weights' other layout) the data gradient
             run_grouped_wgrad  weight and bias gradients; with alpha = -rate and beta = 1 the call
                                is the update of the weights itself
  serving    quantize_rows      the weights once (a scale for each output channel), the activations
                                of each call (a scale for each token)
             run_grouped_i8     the same layer in 8-bit integers, bias and GELU in the epilogue
             quantize_mx        the weights once, the activations of each call straight into the
                                experts' order
             run_grouped_mx     the same layer in MXFP4
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import tiled_matrix_multiply_amd as tmm

BIAS, GELU = tmm.GEMM_EPI_BIAS, tmm.GEMM_EPI_GELU


class Router:
    """The experts of a batch of tokens, two each, and the rows' way to them and back."""

    def __init__(self, handle, scores, top=2):
        tokens, experts = scores.shape
        self.h, self.tokens, self.top, self.rows = handle, tokens, top, tokens * top
        self.expert, self.place = (torch.empty(tokens, top, dtype=torch.int32, device="cuda") for _ in range(2))
        self.weight = torch.empty(tokens, top, device="cuda")
        self.offsets = torch.empty(experts + 1, dtype=torch.int64, device="cuda")
        workspace = torch.empty(tmm.route_workspace_bytes(tokens, experts), dtype=torch.uint8, device="cuda")
        handle.route(scores, self.expert, self.weight, self.place, self.offsets, tokens=tokens, experts=experts,
                     top=top, renorm=True, workspace=workspace)

    def dispatch(self, x, dtype):
        y = torch.empty(self.rows, x.shape[1], device="cuda", dtype=x.dtype)
        self.h.dispatch_rows(x, self.place, y, tokens=self.tokens, top=self.top, K=x.shape[1], rows=self.rows,
                             dtype=dtype)
        return y

    def combine(self, y):
        c = torch.empty(self.tokens, y.shape[1], device="cuda", dtype=y.dtype)
        self.h.combine_rows(y, self.place, c, tokens=self.tokens, top=self.top, K=y.shape[1], rows=self.rows,
                            weight=self.weight)
        return c


def sort_by_expert(scores, experts, top=2):
    """The same in plain operations.  Rows of the sorted batch: the token of each, its weight, and the
    groups' offsets (int64)."""
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


class Layer4:
    """The trained layer in MXFP4."""

    def __init__(self, layer):
        self.h, self.experts = layer.h, layer.experts
        self.b1, self.b2 = layer.b1, layer.b2
        self.w1, self.s1 = self.blocks(layer.w1)
        self.w2, self.s2 = self.blocks(layer.w2)

    def blocks(self, x, place=None, top=1):
        """The rows of x in MXFP4, or with place the rows of the experts' order: elements, scale bytes (whole
        16 to a row, as the tiled kernels need them)."""
        k = x.shape[-1]
        m = x.numel() // k
        q = torch.empty(*x.shape[:-2], x.shape[-2] * top, k // 2, device="cuda", dtype=torch.uint8)
        s = torch.empty(*q.shape[:-1], (k // 32 + 15) // 16 * 16, device="cuda", dtype=torch.uint8)
        self.h.quantize_mx(x, q, s, M=m, K=k, place=place, top=top, rows=m * top, lds=s.shape[-1])
        return q, s

    def product(self, x, w, sw, bias, offsets, epilogue, place=None, top=1):
        q, s = self.blocks(x, place, top)
        y = torch.empty(q.shape[0], w.shape[1], device="cuda", dtype=x.dtype)
        self.h.run_grouped_mx(q, s, w, sw, y, offsets, groups=self.experts, M=q.shape[0], N=w.shape[1], K=x.shape[1],
                              epilogue=epilogue, bias=bias, ldsa=s.shape[1], ldsb=sw.shape[2])
        return y

    def forward(self, x, router):
        """Of the tokens, not of the sorted rows."""
        h = self.product(x, self.w1, self.s1, self.b1, router.offsets, BIAS | GELU, router.place, router.top)
        return self.product(h, self.w2, self.s2, self.b2, router.offsets, BIAS)


def main(tokens=512, dim=256, hidden=768, experts=8, steps=40, rate=1e-4, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    with tmm.Gemm(0) as handle:
        layer = Layer(handle, experts, dim, hidden, gen)
        x = torch.randn(tokens, dim, device="cuda", generator=gen).to(torch.bfloat16)
        scores = torch.randn(tokens, experts, device="cuda", generator=gen)
        router = Router(handle, scores)
        rows, offsets = router.dispatch(x, "bf16"), router.offsets
        target = router.dispatch(torch.randn(tokens, dim, device="cuda", generator=gen), "f32")
        losses = [layer.train_step(rows, target, offsets, rate) for _ in range(steps)]

        y16 = router.combine(layer.forward(rows, offsets)).float()
        y8 = router.combine(Layer8(layer).forward(rows, offsets)).float()
        y4 = router.combine(Layer4(layer).forward(x, router)).float()
        off, off4 = (((y - y16).norm() / y16.norm()).item() for y in (y8, y4))
        losses = [l.item() for l in losses]
        print(f"loss a row: {losses[0]:.2f} -> {losses[-1]:.2f} in {steps} steps; "
              f"8-bit output within {100 * off:.2f}% of the bf16 one, MXFP4 within {100 * off4:.1f}%")
        return losses, off


if __name__ == "__main__":
    main()
