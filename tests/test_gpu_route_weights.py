"""The router's weights within the bound that the header states: (32 + |x - m|) 2^-24 of the weight, x the
expert's logit and m the token's largest, where the scores are at least 2^-125.

In units of 2^-24 of the weight: the argument x - m is rounded once, which is |x - m| of the result; the
exponential is within 2 and its correction adds 1; the sum over up to 1024 experts adds those of its terms
weighted by themselves, at most ln 1024 = 7 for the arguments (the mean of ln(sum / term) is an entropy less
ln(sum)), 2 for the function, and 10 additions in a row; quotient and scale 2.  A sigmoid has no rounded
argument, but one more sum and a reciprocal within 2.

An exponential under 2^-126 is 0.  A sigmoid's part in a renormalised weight is exp(x - m) / (1 + exp(x)) with
m = min(largest, 0), between half the score and the score relative to the largest one: so scores from 2^-125 on
count."""
import numpy as np
import pytest

from test_gpu_experts import RNG, call_route, g, log_scores, scores  # noqa: F401

pytestmark = pytest.mark.gpu


def check_weights(g, x, k, t, kind, renorm, scale, bias=None):  # noqa: F811
    (expert, weight, _, _), x = call_route(g, x, k, t, kind=kind, renorm=renorm, scale=scale, bias=bias)
    rows = np.arange(len(x))[:, None]
    assert (expert >= 0).all()
    if renorm:
        l = log_scores(x, kind)[rows, expert]
        s = np.exp(l - l.max(axis=1, keepdims=True))
        w = s / s.sum(axis=1, keepdims=True)
    else:
        w = s = scores(x, kind)[rows, expert]
    w = scale * w
    away = x.max(axis=1, keepdims=True) - x[rows, expert]
    # (a score within a rounding of the border may be on either side)
    small = s < 2.0 ** -125 * (1 + 2.0 ** -16)
    over = np.abs(weight - w) - ((32 + away) * 2.0 ** -24 * w + np.where(small, scale * 2.0 ** -124, 0.0))
    assert (over <= 0).all(), (x.shape, k, t, kind, renorm, float((over / np.maximum(w, 1e-30)).max()))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_route_weights(g, t, kind, renorm):  # noqa: F811
    """Logits near each other and far apart, near 0 and at the end of the normal numbers of their scores."""
    for E, k in ((2, 2), (16, 16), (60, 4), (128, 8), (256, 16), (300, 32), (1024, 8)):
        for n in (3, 40, 300):
            print(f"[weights] {t} {kind} {renorm} {E} {k} {n}", flush=True)
            rng = RNG([E, n])
            z = rng.standard_normal((n, E))
            for x in (1.5 * z, 20 * z, 40 * rng.random((n, E)), -60 - 30 * rng.random((n, E)), -86 + 2 * rng.random((n, E)),
                      -100 * rng.random((n, E)), 500 + 100 * rng.random((n, E))):
                check_weights(g, x, k, t, kind, renorm, 2.5)
    # choices that a bias takes far below the largest logit
    x = -90 * RNG(1).random((200, 64))
    for k in (1, 7):
        bias = np.where(np.arange(64) % 5 == 0, 3.0, 0.0)
        check_weights(g, x, k, t, kind, renorm, 1.0, bias)
