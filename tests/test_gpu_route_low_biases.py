"""The router with biases of fp32's lowest and highest numbers: other than -infinity they leave an expert
eligible, behind all others, and a run of them worth a number.  Choices, places and offsets have to be equal to
those of the definition in 64 bits."""
import numpy as np
import pytest

from test_gpu_experts import INF, RNG, check_route, g, logits  # noqa: F401

pytestmark = pytest.mark.gpu

LOW = -3.4028234663852886e38


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,best,k", [(8, 2, 1, 4), (16, 4, 3, 6), (64, 16, 12, 3), (60, 4, 2, 5), (128, 16, 9, 15),
                                             (256, 8, 4, 8), (256, 64, 40, 16), (512, 8, 5, 8), (600, 4, 2, 20), (1023, 33, 20, 7)])
def test_route_biases_at_the_ends(g, kind, E, groups, best, k):  # noqa: F811
    rng = RNG([E, groups])
    some = 0.1 * rng.standard_normal(E)
    mixed = np.where(rng.random(E) < 0.7, LOW, some)
    runs = np.where(np.arange(E) * groups // E % 2 == 0, LOW, some)          # whole runs
    few = np.full(E, -INF)
    few[rng.permutation(E)[:max(2, E // 8)]] = LOW                          # fewer than asked for, and these low
    for name, bias in (("all low", np.full(E, LOW)), ("mixed", mixed), ("runs", runs), ("few", few), ("high", -mixed),
                       ("both", np.where(rng.random(E) < 0.5, LOW, -LOW)), ("near low", LOW * (1 - 1e-6 * rng.random(E)))):
        for n in (3, 40, 150):
            x = logits(n, E, k)
            x[0, ::3] = -INF
            print(f"[route] {name} {kind} {E} {groups} {n}", flush=True)
            for of in (1, 2):
                check_route(g, x, k, "f32", kind=kind, bias=bias, groups=groups, best=best, of=of, renorm=n == 40)
            check_route(g, x, k, "bf16", kind=kind, bias=bias)
