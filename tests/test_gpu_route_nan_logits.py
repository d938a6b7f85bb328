"""A NaN logit in the router where the experts of a lane are all NaN: the choice is that of the definition (a
key that is NaN counts as +infinity), for every place of the NaN, with keys below 0.

Choices, places and offsets have to be equal; the weights' bounds are test_gpu_experts.py's."""
import numpy as np
import pytest

from test_gpu_experts import INF, NAN, RNG, call_grad, check_route, g, logits  # noqa: F401

pytestmark = pytest.mark.gpu


# (experts, the run of neighbours that are NaN: as many as a lane holds)
@pytest.mark.parametrize("E,run", [(2, 1), (8, 1), (16, 1), (64, 4), (60, 4), (128, 8), (256, 16), (256, 4), (512, 8), (1024, 16)])
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_route_nan_at_each_expert(g, kind, E, run):  # noqa: F811
    """Every aligned run of a lane's experts in turn, with a bias that makes the other keys negative.  The same
    tokens alone and in a batch: a few tokens have other lanes than many."""
    x = logits(E // run + 5, E, run)
    for i in range(E // run):
        x[i, i * run:(i + 1) * run] = NAN
    x[-1], x[-2], x[-3] = NAN, -INF, np.where(np.arange(E) % 3 == 0, NAN, -INF)
    x[-4, ::2] = NAN
    x = x[RNG(E).permutation(len(x))]
    bias = -2 + 0.1 * RNG([E, run]).standard_normal(E)
    for k in sorted({1, 2, 4, 8, 16, min(E, 20)}):
        if k > E:
            continue
        print(f"[route] NaN {kind} {E} {run} {k}", flush=True)
        for renorm in (False, True):
            check_route(g, x, k, "f32", kind=kind, bias=bias, renorm=renorm)
        check_route(g, x[:5], k, "bf16", kind=kind, bias=bias)
        check_route(g, np.concatenate([x] * (1 + 70 // len(x))), k, "f16", kind=kind, bias=bias)
        check_route(g, x, k, "f32", kind=kind)
    for groups, best in ((2, 1), (4, 2)):
        if E % groups == 0:
            for of in (1, 2):
                check_route(g, x, min(4, best * E // groups), "f32", kind=kind, bias=bias, groups=groups, best=best, of=of)


@pytest.mark.parametrize("E,groups,best", [(8, 1, 1), (16, 4, 2), (60, 1, 1), (256, 8, 3), (512, 1, 1)])
def test_route_softmax_of_nan_is_not_silent(g, E, groups, best):  # noqa: F811
    """A softmax over NaN or +infinity has no numbers, so that no expert's weight is one, renormalised or not,
    also where the expert with the NaN is not among the chosen."""
    for n in (4, 40, 150):
        x = logits(n, E, n)
        for t, (e, v) in enumerate([(E - 1, NAN), (0, NAN), (E // 2, INF)]):
            x[t, e] = v
        bias = 0.1 * RNG(E).standard_normal(E)
        bias[E - 1] = -INF
        for b, of in ((bias, 1), (bias, 2), (None, 2)):
            for renorm in (False, True):
                print(f"[route] NaN softmax {E} {groups} {n} {b is not None} {of} {renorm}", flush=True)
                with np.errstate(invalid="ignore"):
                    _, weight, _, _ = check_route(g, x, 2, "f32", kind="softmax", bias=b, groups=groups, best=best, of=of,
                                                  renorm=renorm)
                assert np.isnan(weight[:3]).all() and np.isfinite(weight[3:]).all()


@pytest.mark.parametrize("E,k", [(8, 2), (60, 4), (200, 16), (300, 6)])
def test_route_grad_of_nan(g, E, k):  # noqa: F811
    """What NaN and +infinity among the logits reach: of a softmax as it is every gradient of the token, with
    renormalisation those of the chosen if it is one of them; of a sigmoid the expert's own, or those of the
    chosen."""
    rng = RNG([E, k])
    n = 20
    x = logits(n, E, 3)
    expert = np.argsort(rng.random((n, E)), axis=1)[:, :k]
    x[1, expert[1, 0]], x[3, expert[3, k - 1]] = NAN, INF
    free = [next(e for e in range(E) if e not in expert[t]) for t in range(n)]
    x[5, free[5]], x[7, free[7]] = NAN, INF
    dw = rng.standard_normal((n, k))
    chosen = np.zeros((n, E), dtype=bool)
    chosen[np.arange(n)[:, None], expert] = True
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            got, _ = call_grad(g, x, expert, dw, "f32", kind, renorm, 1.5)
            want = np.zeros((n, E), dtype=bool)
            if kind == "softmax" and not renorm:
                want[[1, 3, 5, 7]] = True
            elif renorm:
                want[1] = chosen[1]
                want[3] = chosen[3] & (kind == "softmax")
            else:
                want[1, expert[1, 0]] = True
            assert np.array_equal(np.isnan(got), want), (kind, renorm)
            if kind == "sigmoid" or renorm:
                assert (got[~chosen & ~want] == 0).all()
