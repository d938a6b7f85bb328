"""examples/moe_layer.py: the layer learns, its gradients agree with autograd's, and the 8-bit layer
answers as the 16-bit one does."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_trains_and_serves(moe):
    losses, off = moe.main(steps=30)
    assert losses[-1] < 0.9 * losses[0]
    # codes are off by at most half of 1/127 of a row's largest value, for activations and weights
    # in two layers: a few percent of the typical value
    assert 0 < off < 0.05


def test_update_is_the_gradient(moe):
    """One step's change of the weights against autograd of the plain layer in fp32 on the CPU."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    gen = torch.Generator(device="cuda").manual_seed(3)
    with tmm.Gemm(0) as handle:
        layer = moe.Layer(handle, 4, 64, 96, gen)
        x = torch.randn(60, 64, device="cuda", generator=gen).to(torch.bfloat16)
        token, _, offsets = moe.sort_by_expert(torch.randn(60, 4, device="cuda", generator=gen), 4)
        rows, target = x[token], torch.randn(120, 64, device="cuda", generator=gen)
        params = [p.float().cpu().requires_grad_() for p in (layer.w1, layer.w2, layer.b1, layer.b2)]
        w1, w2, b1, b2 = params
        off, r, t = offsets.tolist(), rows.float().cpu(), target.cpu()
        assert off[0] == 0 and off[-1] == 120
        loss = 0.0
        for e in range(4):
            cut = slice(off[e], off[e + 1])
            h = torch.nn.functional.gelu(r[cut] @ w1[e].t() + b1[e])
            loss = loss + 0.5 * ((h @ w2[e].t() + b2[e] - t[cut]) ** 2).sum()
        loss.backward()
        before = [p.clone() for p in (layer.w1, layer.w2, layer.b1, layer.b2)]
        rate = 0.25
        layer.train_step(rows, target, offsets, rate)
        for p, old, ref in zip((layer.w1, layer.w2, layer.b1, layer.b2), before, params):
            step = (old.float() - p.float()).cpu() / rate
            # bf16 activations and gradients on the way, and the weight rounded to bf16 at the end
            assert (step - ref.grad).norm() < 0.02 * ref.grad.norm()
