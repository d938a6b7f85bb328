"""Near and equal keys in the router: chosen as 64 bits order them, whatever else is in the same wave.

Every choice, place and offset has to be that of the definition in 64 bits, ties to the lower expert; the
weights' bounds are test_gpu_experts.py's."""
import numpy as np
import pytest

from test_gpu_experts import RNG, check_route, g  # noqa: F401

pytestmark = pytest.mark.gpu


def close_logits(n, E, k, seed, top=2):
    """fp32 logits from `top` down whose keys differ in their last four bits, in all the places that matter: tokens of all
    kinds in any order, so that every two of them meet in a wave.  Kinds: neighbours clearly apart; one near pair
    among the chosen; one at the border of the choice; near pairs at the head and at the border; many near
    keys around the border; near keys everywhere."""
    rng = RNG([n, E, k, seed])
    x = np.empty((n, E), dtype=np.float32)
    for t in range(n):
        v = (top - np.arange(E) / E).astype(np.float32)          # falling, far apart
        kind = rng.integers(6)
        ulps = rng.integers(-12, 13, E).astype(np.float32) * np.float32(2.0 ** -23)
        near = []
        if kind in (1, 3):
            near.append((0, 2))
        if kind in (2, 3):
            near.append((k - 1, k + 1))
        if kind == 4:
            near.append((max(0, k - 5), k + 1 + rng.integers(12)))
        if kind == 5:
            near.append((0, E))
        for lo, hi in near:
            v[lo:hi] = v[lo] + ulps[lo:hi]
        x[t, rng.permutation(E)] = v
    return x.astype(np.float64)


@pytest.mark.parametrize("E", [17, 64, 128, 256, 300, 600])
def test_route_near_logits(g, E):  # noqa: F811
    """Choices of up to as many experts as a token has lanes, and more."""
    for k in (1, 4, 8, 12, 13, 14, 15, 16, 17, 32):
        if k > E:
            continue
        for n in (1, 4, 16, 23, 64, 301):
            print(f"[route] near {E} {k} {n}", flush=True)
            for top in (2, -1):                      # positive and negative logits
                check_route(g, close_logits(n, E, k, 1, top), k, "f32", renorm=n % 2 == 0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [17, 64, 128, 256])
def test_route_near_biased_keys(g, kind, E):  # noqa: F811
    """With a bias that is zero, or differs in the last bits of the scores."""
    for k in (12, 14, 15, 16):
        for n in (13, 64, 202):
            print(f"[route] near biased {kind} {E} {k} {n}", flush=True)
            rng = RNG([E, k, n])
            x = close_logits(n, E, k, 2)
            check_route(g, x, k, "f32", kind=kind, bias=np.zeros(E))
            check_route(g, x, k, "f32", kind=kind, bias=1e-7 * rng.standard_normal(E), renorm=True)
            check_route(g, 4 * x, k, "f32", kind=kind, bias=-1 + 1e-6 * rng.standard_normal(E))
            if E % 4 == 0:
                check_route(g, x, k, "f32", kind=kind, bias=1e-7 * rng.standard_normal(E), groups=4, best=3, of=2)
                check_route(g, x, k, "f32", kind=kind, groups=4, best=3, of=2)


def test_route_scores_below_the_normal_numbers(g):  # noqa: F811
    """Sigmoid scores under 2^-126 with biases of their size: the sums are compared as 64 bits have them."""
    rng = RNG(7)
    for E, k in ((8, 3), (16, 16), (60, 6), (256, 16), (600, 20)):
        for n in (3, 40, 150):
            x = -(86 + 4 * rng.random((n, E)))
            x[0] = -100 - rng.random(E)
            x[1] = -700 - 10 * rng.random(E)
            bias = (4e-39 * rng.random(E)).astype(np.float32).astype(np.float64)
            print(f"[route] tiny {E} {k} {n}", flush=True)
            check_route(g, x, k, "f32", kind="sigmoid", bias=bias)
            check_route(g, x, k, "f32", kind="sigmoid", bias=np.zeros(E))
            if E % 4 == 0:
                check_route(g, x, min(k, 3 * E // 4), "f32", kind="sigmoid", bias=bias, groups=4, best=3, of=2)
