"""Routing to experts, the rows' way there and back, and products by expert in MXFP4 on the GPU, against
plain numpy in 64 bits.

Tolerances (fixed before the first run).
  weights: the argument of an exponential is rounded once (|x - m| 2^-24, which is that much of its
    result), the function is within 2^-23, the quotients and products of a weight are six more fp32
    roundings or less: (16 + |x - m|) 2^-24 of the weight, twice that where a sum over the chosen goes in.
  gradients: the same of sum |terms| for each of two weights in a term, plus sums of up to E
    positive fp32 terms over lanes (24 roundings), plus half a step of the result's type.
  sums of products: n fp32 roundings of sum |a b|, plus half a step.  A product of MXFP4 is exact; fp32
    sums in any order stay within K 2^-23 of sum |a b|, the epilogue adds 4 (20 with GELU) roundings.
Choices, places, offsets, codes and scales have to be equal.
"""
import numpy as np
import pytest
from scipy.special import erfc

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
U32 = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
RNG = np.random.default_rng


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tiled_matrix_multiply_amd as tmm
    h = tmm.Gemm(0)
    yield h
    h.close()


def T():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")
    return t if dtype is None else t.to(T()[dtype])


def host(t):
    return t.double().cpu().numpy()


def bits(t):
    import torch
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def check(got, ref, lim, c_type, what):
    """|got - ref| <= lim, and infinities and NaN where the reference has them.  From 65520 = 65504 + half
    a step on, round to nearest even gives fp16's infinity: where the reference is within its bound of
    that, infinity of its sign is the rounded value of a number within the bound."""
    fin = np.isfinite(ref)
    if c_type == "f16":
        over = fin & (np.abs(ref) + lim >= 65520) & np.isinf(got) & (np.sign(got) == np.sign(ref))
        got = np.where(over, ref, got)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), what
    err = np.abs(got[fin] - ref[fin]) - TINY[c_type]
    bad = ~(err <= lim[fin])
    assert not bad.any(), (what, int(bad.sum()), float((err - lim[fin]).max()))


# -------------------------------------------------------------------------------- route --

def scores(x, kind):
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = np.max(x, axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        return e / e.sum(axis=1, keepdims=True)


def log_scores(x, kind):
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if kind == "sigmoid":
            return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
        top = np.max(x, axis=1, keepdims=True)
        return x - np.where(np.isneginf(top), 0.0, top)


def reference(x, k, kind, bias, groups, best, of, renorm, scale):
    """expert, weight (64 bits), place and offsets, one token at a time."""
    n, E = x.shape
    s, ls = scores(x, kind), log_scores(x, kind)
    expert = np.full((n, k), -1, dtype=np.int64)
    weight = np.zeros((n, k))
    size = E // groups
    for t in range(n):
        off = np.isneginf(x[t])
        key = x[t].copy()
        worth = x[t].copy() if of == 1 else s[t].copy()
        if bias is not None:
            key = s[t] + bias
            off = off | np.isneginf(bias)
            worth = key.copy()
        key[np.isnan(key)], worth[np.isnan(worth)] = INF, INF
        key[off], worth[off] = -INF, -INF
        if groups > 1:
            total = np.full(groups, -INF)
            for q in range(groups):
                w = np.sort(worth[q * size:(q + 1) * size])[::-1][:of]
                w = w[~np.isneginf(w)]
                if w.size:
                    total[q] = w.sum()
            kept = [q for q in np.argsort(-total, kind="stable")[:best] if total[q] != -INF]
            drop = np.ones(E, dtype=bool)
            for q in kept:
                drop[q * size:(q + 1) * size] = False
            key[drop] = -INF
        order = [e for e in np.argsort(-key, kind="stable")[:k] if key[e] != -INF]
        expert[t, :len(order)] = order
        if order:
            if renorm:
                l = ls[t, order]
                with np.errstate(invalid="ignore"):
                    w = np.exp(l - (INF if np.isnan(l).any() else l.max()))
                w = np.full(len(order), NAN) if np.isnan(l).any() else w / w.sum()
            else:
                w = s[t, order]
            weight[t, :len(order)] = scale * w
    flat = expert.ravel()
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    place = np.empty(flat.size, dtype=np.int64)
    place[order] = np.arange(flat.size)
    place[flat < 0] = -1
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))])
    return expert, weight, place.reshape(n, k), offsets


def call_route(g, x, k, t="f32", *, kind="softmax", bias=None, groups=1, best=1, of=1, renorm=False,
               scale=1.0, ldl=None, stream=None):
    """The call on a host matrix (after its rounding to t): the results on the host, and the rounded x."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    n, E = x.shape
    ldl = ldl or E
    X = torch.full((max(n, 1), ldl), NAN, device="cuda:0", dtype=T()[t])
    if n:
        X[:, :E] = dev(x, t)
    out = [torch.full((n, k), 7, dtype=torch.int32, device="cuda:0"),
           torch.full((n, k), NAN, device="cuda:0"),
           torch.full((n, k), 7, dtype=torch.int32, device="cuda:0"),
           torch.full((E + 1,), 7, dtype=torch.int64, device="cuda:0")]
    nb = tmm.route_workspace_bytes(n, E)
    ws = torch.full((nb + 16,), 255, dtype=torch.uint8, device="cuda:0")
    b = None if bias is None else dev(bias.astype(np.float32))
    g.route(X, *out, tokens=n, experts=E, top=k, x_type=t, score=kind, bias=b, groups=groups, top_groups=best,
            group_top=of, renorm=renorm, scale=scale, ldl=ldl, workspace=ws, workspace_bytes=nb, stream=stream)
    torch.cuda.synchronize()
    assert (ws[nb:] == 255).all()
    return [o.cpu().numpy() for o in out], host(X[:n, :E])


def check_route(g, x, k, t="f32", **kw):
    (expert, weight, place, offsets), x = call_route(g, x, k, t, **kw)
    kw.pop("ldl", None)
    kind, bias = kw.get("kind", "softmax"), kw.get("bias")
    ref = reference(x, k, kind, None if bias is None else bias.astype(np.float32).astype(np.float64),
                    kw.get("groups", 1), kw.get("best", 1), kw.get("of", 1), kw.get("renorm", False),
                    kw.get("scale", 1.0))
    what = (x.shape, k, t, {a: b for a, b in kw.items() if a != "bias"}, bias is not None)
    assert np.array_equal(expert, ref[0]), what
    assert np.array_equal(place, ref[2]), what
    assert np.array_equal(offsets, ref[3]), what
    fin = np.where(np.isfinite(x), x, 0.0)
    span = np.minimum(fin.max(axis=1) - fin.min(axis=1), 200.0) if x.size else np.zeros(len(x))
    check(weight.astype(np.float64), ref[1], 2 * (16 + span)[:, None] * U32 * np.abs(ref[1]) + 1e-37, "f32", what)
    return ref


def logits(n, E, seed, spread=1.5):
    rng = RNG([n, E, seed])
    return spread * rng.standard_normal((n, E)) + 0.5 * rng.standard_normal(E)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_route_sizes(g, t, kind):
    for i, n in enumerate([1, 2, 15, 16, 17, 63, 64, 65, 200, 1037]):
        for j, (E, k) in enumerate([(1, 1), (2, 2), (7, 3), (16, 16), (17, 2), (60, 4), (64, 32), (65, 8), (128, 8),
                                    (256, 8), (257, 5), (1024, 32)]):
            if n * E > 300000 and (i + j) % 2:
                continue
            print(f"[route] {t} {kind} {n} {E} {k}", flush=True)
            bias = 0.2 * RNG([i, j]).standard_normal(E) if (i + j) % 2 else None
            check_route(g, logits(n, E, i + j), k, t, kind=kind, bias=bias, renorm=(i + j) % 3 == 0,
                        scale=2.5 if i % 2 else 1.0, ldl=E + 3 if j % 2 else None)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("of", [1, 2])
def test_route_groups(g, kind, of):
    for i, (E, groups, best, k) in enumerate([(256, 8, 4, 8), (64, 8, 2, 4), (60, 4, 3, 4), (64, 64, 6, 6), (12, 3, 1, 4),
                                              (1024, 32, 5, 16), (1000, 8, 8, 8), (16, 16, 1, 1), (192, 6, 2, 8),
                                              (512, 2, 1, 32), (640, 5, 3, 7), (48, 24, 9, 3)]):
        for n in (1, 33, 300):
            for b in (False, True):
                print(f"[route] groups {kind} {of} {E} {groups} {best} {k} {n} {b}", flush=True)
                bias = 0.3 * RNG([i, n]).standard_normal(E) if b else None
                check_route(g, logits(n, E, i), k, "bf16" if b else "f32", kind=kind, bias=bias, groups=groups,
                            best=best, of=of, renorm=i % 2 == 0, scale=1.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_what_is_not_there(g, kind):
    """Rows without an expert, with fewer than asked for, experts that a bias takes out, the lowest
    numbers of a type, infinities and NaN."""
    for t, low in (("f32", -3.4028234663852886e38), ("bf16", -3.3895313892515355e38), ("f16", -65504.0)):
        for n in (40, 150):
            for E, groups, best in ((24, 1, 1), (24, 4, 2), (200, 1, 1), (200, 8, 3), (600, 4, 2)):
                x = logits(n, E, 5)
                x[0] = -INF                       # padding
                x[1, 1:] = -INF                   # one expert left
                x[2] = low
                x[3] = low
                x[3, E // 2] = 0.0
                x[4, ::2] = -INF
                x[5, :E // 2] = -INF
                x[6] = 0.0                        # all equal
                x[7] = np.round(x[7])             # many equal
                x[n - 3:] = -INF
                bias = 0.1 * RNG(9).standard_normal(E)
                bias[1] = -INF
                for b in (None, bias):
                    for renorm in (False, True):
                        print(f"[route] masks {kind} {t} {n} {E} {groups} {renorm} {b is not None}", flush=True)
                        for of in (1, 2):
                            check_route(g, x, 4, t, kind=kind, bias=b, groups=groups, best=best, of=of, renorm=renorm)


def test_route_nan_and_infinity_are_not_silent(g):
    x = logits(8, 32, 1)
    x[0] = NAN
    x[1, 20] = NAN
    x[2, 3] = INF
    x[3, 3], x[3, 9] = INF, NAN
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            (expert, weight, _, _), _ = call_route(g, x, 4, "f32", kind=kind, renorm=renorm)
            assert expert[0].tolist() == [0, 1, 2, 3] and np.isnan(weight[0]).all()
            assert expert[1, 0] == 20 and np.isnan(weight[1, 0])
            assert expert[2, 0] == 3 and expert[3, :2].tolist() == [3, 9] and np.isnan(weight[3, 1])
            if renorm or kind == "softmax":
                assert np.isnan(weight[1]).all()
            assert np.isfinite(weight[4:]).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_nan_in_masked_places(g, kind):
    """An expert that a bias of -infinity takes out stays out whatever its logit: NaN, infinity; in a
    softmax these make every score NaN, and the experts that are left come in their order."""
    for E, groups, best in ((32, 1, 1), (32, 4, 2), (200, 1, 1), (300, 1, 1)):
        for n in (3, 20):
            x = logits(n, E, E)
            x[0, 5] = NAN
            x[1, 5], x[1, 9] = INF, NAN
            x[2, 9] = NAN
            bias = 0.1 * RNG(E).standard_normal(E)
            bias[5] = bias[9] = -INF
            for renorm in (False, True):
                (expert, weight, place, _), _ = call_route(g, x, 4, "f32", kind=kind, bias=bias, groups=groups, best=best,
                                                           renorm=renorm)
                assert not np.isin(expert, [5, 9]).any() and (expert >= 0).all() and (place >= 0).all(), (E, groups, n)
                if kind == "sigmoid":
                    ref = reference(np.where(np.isin(np.arange(E), [5, 9]), -INF, x.astype(np.float32).astype(np.float64)), 4,
                                    kind, bias.astype(np.float32).astype(np.float64), groups, best, 1, renorm, 1.0)
                    assert np.array_equal(expert, ref[0]) and np.isfinite(weight).all()
                else:
                    first = [e for e in range(E) if e not in (5, 9)][:4]
                    assert all(expert[t].tolist() == first for t in range(3))


def test_route_close_keys(g):
    """Keys that fp32 cannot tell apart are ordered as 64 bits order them."""
    E, n = 128, 400
    rng = RNG(11)
    x = np.float32(rng.standard_normal((n, 1))) + np.float32(1e-6) * rng.integers(-3, 4, (n, E)).astype(np.float32)
    bias = (1e-7 * rng.standard_normal(E)).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        check_route(g, x.astype(np.float64), 8, "f32", kind=kind, bias=bias)
        check_route(g, x.astype(np.float64), 8, "f32", kind=kind, bias=bias, groups=8, best=3, of=2)
        check_route(g, x.astype(np.float64), 8, "f32", kind=kind, groups=8, best=3, of=2)
    big = 20 + 10 * rng.standard_normal((n, E))            # scores near 1 next to each other
    check_route(g, big, 8, "bf16", kind="sigmoid", bias=bias)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_many_experts(g, kind):
    """More than 256 experts, eight to a lane, around the borders of the tokens to a workgroup."""
    for i, n in enumerate([3, 66, 256, 257, 400, 512, 513]):
        for j, (E, groups, best, k) in enumerate([(300, 1, 1, 4), (512, 1, 1, 8), (512, 8, 3, 8), (416, 4, 2, 32), (513, 1, 1, 6)]):
            print(f"[route] many {kind} {n} {E} {groups} {k}", flush=True)
            x = logits(n, E, i + j)
            x[n // 2] = -INF
            x[n - 1, 7:] = -INF
            x[0] = np.float32(0.5) + np.float32(1e-6) * RNG([i, j]).integers(-2, 3, E)     # close and equal keys
            x = x.astype(np.float32).astype(np.float64)
            bias = 0.2 * RNG([i, j]).standard_normal(E) if (i + j) % 2 else None
            check_route(g, x, k, "f32", kind=kind, bias=bias, groups=groups, best=best, of=1 + j % 2, renorm=i % 2 == 0)


def test_route_no_tokens_and_many(g):
    import torch
    _, _, _, offsets = call_route(g, np.zeros((0, 5)), 2)[0]
    assert (offsets == 0).all()
    # 70000 tokens: blocks of 64, several to a workgroup of the second kernel
    x = dev(logits(70000, 24, 3), "bf16")
    import tiled_matrix_multiply_amd as tmm
    e, p = (torch.empty(70000, 3, dtype=torch.int32, device="cuda:0") for _ in range(2))
    w, o = torch.empty(70000, 3, device="cuda:0"), torch.empty(25, dtype=torch.int64, device="cuda:0")
    ws = torch.empty(tmm.route_workspace_bytes(70000, 24), dtype=torch.uint8, device="cuda:0")
    g.route(x, e, w, p, o, tokens=70000, experts=24, top=3, x_type="bf16", workspace=ws)
    key, at = x.double().cpu().sort(dim=1, descending=True, stable=True)
    assert torch.equal(e.cpu().long(), at[:, :3])
    flat = e.cpu().long().flatten()
    order = torch.argsort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel())
    assert torch.equal(p.cpu().long().flatten(), place)
    assert torch.equal(o.cpu(), torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(flat, minlength=24).cumsum(0)]))


# ----------------------------------------------------------------------- route's gradient --

def weights_64(x, expert, kind, renorm, scale):
    """The weights of given choices in 64 bits (-1: 0)."""
    s = scores(x, kind)
    rows = np.arange(len(x))[:, None]
    w = np.where(expert >= 0, s[rows, np.maximum(expert, 0)], 0.0)
    return scale * (w / w.sum(axis=1, keepdims=True) if renorm else w)


def grad_reference(x, expert, dw, kind, renorm, scale):
    """The formula, and the sum of the sizes of its terms."""
    n, E = x.shape
    s = scores(x, kind)
    rows = np.arange(n)[:, None]
    there = expert >= 0
    at = np.maximum(expert, 0)
    sj = np.where(there, s[rows, at], 0.0)
    gj = np.where(there, scale * dw, 0.0)
    w = sj / np.maximum(sj.sum(axis=1, keepdims=True), 1e-300) if renorm else sj
    d = w * (gj - (w * gj).sum(axis=1, keepdims=True)) if renorm else w * gj
    size = w * (np.abs(gj) + (w * np.abs(gj)).sum(axis=1, keepdims=True)) if renorm else np.abs(d)
    dx, den = np.zeros((n, E)), np.zeros((n, E))
    for j in range(expert.shape[1]):
        dx[rows[:, 0], at[:, j]] += np.where(there[:, j], d[:, j], 0.0)
        den[rows[:, 0], at[:, j]] += np.where(there[:, j], size[:, j], 0.0)
    if kind == "sigmoid":
        dx, den = dx * (1 - s), den * (1 - s)
    elif not renorm:
        dx, den = dx - s * d.sum(axis=1, keepdims=True), den + s * np.abs(d).sum(axis=1, keepdims=True)
    return dx, den


def call_grad(g, x, expert, dw, t, kind, renorm, scale, ldl=None, ldd=None):
    import torch
    n, E = x.shape
    k = expert.shape[1]
    ldl, ldd = ldl or E, ldd or E
    X = torch.full((n, ldl), NAN, device="cuda:0", dtype=T()[t])
    X[:, :E] = dev(x, t)
    dX = torch.full((n, ldd), 7.0, device="cuda:0", dtype=T()[t])
    g.route_grad(X, dev(expert.astype(np.int32)), dev(dw.astype(np.float32)), dX, tokens=n, experts=E, top=k,
                 x_type=t, score=kind, renorm=renorm, scale=scale, ldl=ldl, ldd=ldd)
    torch.cuda.synchronize()
    assert (dX[:, E:] == 7.0).all()
    return host(dX[:, :E]), host(X[:, :E])


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_route_grad(g, t, kind, renorm):
    for i, n in enumerate([1, 5, 16, 17, 130]):
        for j, (E, k) in enumerate([(1, 1), (3, 2), (16, 16), (33, 4), (64, 32), (200, 8), (256, 17), (300, 6), (1024, 32)]):
            print(f"[route_grad] {t} {kind} {renorm} {n} {E} {k}", flush=True)
            rng = RNG([i, j])
            x = logits(n, E, i + j)
            x[0, 0] = -INF if E > 1 else 0.5
            expert = np.argsort(rng.random((n, E)), axis=1)[:, :k]
            expert[n // 2, k // 2:] = -1
            if E > 1:
                expert[0][expert[0] == 0] = -1
            dw = rng.standard_normal((n, k)).astype(np.float32).astype(np.float64)
            got, x = call_grad(g, x, expert, dw, t, kind, renorm, 1.25, E + 5 if j % 2 else None, E + 1 if i % 2 else None)
            ref, den = grad_reference(x, expert, dw, kind, renorm, 1.25)
            check(got, ref, (100 + 4 * 12) * U32 * den + HALF_STEP[t] * np.abs(ref), t, (n, E, k))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_grad_against_differences(g, kind, renorm):
    """Central differences of the weights' formula in 64 bits, with the choice held: off by a third
    derivative (below 1 here) times h^2, and rounding of 1e-16 / h."""
    rng = RNG(3)
    n, E, k, h = 12, 20, 4, 1e-4
    x = logits(n, E, 2).astype(np.float32).astype(np.float64)
    expert = reference(x, k, kind, None, 1, 1, 1, renorm, 1.0)[0]
    dw = rng.standard_normal((n, k)).astype(np.float32).astype(np.float64)
    got, _ = call_grad(g, x, expert, dw, "f32", kind, renorm, 2.0)
    for e in range(E):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        f = [(dw * weights_64(v, expert, kind, renorm, 2.0)).sum(axis=1) for v in (up, down)]
        diff = (f[0] - f[1]) / (2 * h)
        assert np.abs(got[:, e] - diff).max() <= 2 * np.abs(dw).sum(axis=1).max() * (h * h + 150 * U32), e


def test_route_grad_of_a_weight_near_one(g):
    """No cancellation: the largest logit stands out by 12, so that its weight is 1 to 2^-17."""
    x = logits(16, 64, 8, spread=0.1)
    x[:, 5] = 12.0
    expert = np.tile(np.array([5, 1, 60]), (16, 1))
    dw = RNG(4).standard_normal((16, 3)).astype(np.float32).astype(np.float64)
    for kind, renorm in (("softmax", False), ("softmax", True)):
        got, xr = call_grad(g, x, expert, dw, "f32", kind, renorm, 1.0)
        ref, _ = grad_reference(xr, expert, dw, kind, renorm, 1.0)
        # each term is a product of scores with a difference of two numbers
        assert (np.abs(got - ref)[:, 5] <= 400 * U32 * np.abs(ref[:, 5])).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_grad_of_masked_tokens(g, kind, renorm):
    """Tokens without any logit, with one, and with none but those that were not chosen: no NaN."""
    for E, k in ((5, 2), (60, 4), (256, 8), (300, 20)):
        x = logits(6, E, E)
        expert = np.argsort(RNG(E).random((6, E)), axis=1)[:, :k]
        x[0] = x[1] = x[5] = -INF
        expert[0] = -1                                    # as the router answers; token 1 names experts all the same
        x[2, 1:] = -INF
        expert[2], expert[2, 0] = -1, 0
        expert[3] = -1
        dw = RNG(7).standard_normal((6, k)).astype(np.float32).astype(np.float64)
        got, xr = call_grad(g, x, expert, dw, "f32", kind, renorm, 1.5)
        assert (got[[0, 1, 3, 5]] == 0).all()
        keep = [2, 4]
        with np.errstate(invalid="ignore"):
            ref, den = grad_reference(xr[keep], expert[keep], dw[keep], kind, renorm, 1.5)
        check(got[keep], ref, 148 * U32 * den, "f32", (E, k))


def test_route_grad_skips_what_is_no_expert(g):
    x = logits(4, 10, 1)
    expert = np.array([[1, 2], [-1, 3], [10, 4], [2 ** 31 - 1, -2 ** 31]])
    dw = np.ones((4, 2))
    got, xr = call_grad(g, x, expert, dw, "f32", "sigmoid", False, 1.0)
    ref, _ = grad_reference(xr, np.where((expert < 0) | (expert > 9), -1, expert), dw, "sigmoid", False, 1.0)
    check(got, ref, 148 * U32 * np.abs(ref), "f32", "skips")
    assert (got[3] == 0).all()


# --------------------------------------------------------------------------------- rows --

def places(n, k, rows, seed, skip=0.2):
    """Distinct rows for the pairs, some of them none, some far out."""
    rng = RNG([n, k, seed])
    p = rng.permutation(rows)[:n * k].reshape(n, k).astype(np.int64)
    out = rng.random((n, k)) < skip
    p[out] = rng.choice([-1, rows, -2 ** 31, 2 ** 31 - 1], size=int(out.sum()))
    return p


ROWS = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (16, 2, 2048), (65, 3, 100), (130, 8, 33), (40, 1, 8), (33, 5, 5000),
        (20, 2, 9001), (600, 4, 64)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_dispatch(g, t):
    import torch
    for i, (n, k, K) in enumerate(ROWS):
        print(f"[dispatch] {t} {n} {k} {K}", flush=True)
        R, ldx, lda = n * k + 3, K + i % 3, K + i % 2
        place = places(n, k, R, i)
        X, A = torch.randn(n, ldx, device="cuda:0").to(T()[t]), torch.randn(R, lda, device="cuda:0").to(T()[t])
        X[0, 0] = NAN
        want = A.clone()
        for r in range(n):
            for j in range(k):
                if 0 <= place[r, j] < R:
                    want[place[r, j], :K] = X[r, :K]
        g.dispatch_rows(X, dev(place.astype(np.int32)), A, tokens=n, top=k, K=K, rows=R, dtype=t, ldx=ldx, lda=lda)
        torch.cuda.synchronize()
        assert torch.equal(bits(A), bits(want)), (n, k, K)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("beta", [0.0, 1.0, -0.5])
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_combine(g, t, beta, weighted):
    import torch
    for i, (n, k, K) in enumerate(ROWS):
        print(f"[combine] {t} {beta} {weighted} {n} {k} {K}", flush=True)
        R, ldy, ldc = n * k + 3, K + i % 3, K + i % 2
        place = places(n, k, R, i)
        ok = (place >= 0) & (place < R)
        Y, C = torch.randn(R, ldy, device="cuda:0").to(T()[t]), torch.randn(n, ldc, device="cuda:0").to(T()[t])
        unused = np.ones(R, dtype=bool)
        unused[place[ok]] = False
        Y[torch.from_numpy(unused).cuda()] = NAN
        w = RNG(i).standard_normal((n, k)).astype(np.float32)
        w[~ok] = NAN
        before = C.clone()
        if beta == 0.0:
            C[:, :K] = NAN
        g.combine_rows(Y, dev(place.astype(np.int32)), C, tokens=n, top=k, K=K, rows=R, dtype=t,
                       weight=dev(w) if weighted else None, beta=beta, ldy=ldy, ldc=ldc)
        torch.cuda.synchronize()
        wv = np.where(ok, w.astype(np.float64) if weighted else 1.0, 0.0)
        y = np.where(ok[:, :, None], host(Y)[np.where(ok, place, 0), :K], 0.0)
        ref = (wv[:, :, None] * y).sum(axis=1) + (beta * host(before)[:, :K] if beta else 0.0)
        den = (np.abs(wv)[:, :, None] * np.abs(y)).sum(axis=1) + np.abs(beta * host(before)[:, :K])
        check(host(C)[:, :K], ref, (k + 2) * U32 * den + HALF_STEP[t] * (np.abs(ref) + (k + 2) * U32 * den), t, (n, k, K))
        assert torch.equal(bits(C[:, K:]), bits(before[:, K:]))


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_combine_grad(g, t):
    import torch
    for i, (n, k, K) in enumerate(ROWS):
        print(f"[combine_grad] {t} {n} {k} {K}", flush=True)
        R, ldd, ldy, lddy = n * k + 3, K + i % 3, K + i % 2, K + (i + 1) % 3
        place = places(n, k, R, i)
        ok = (place >= 0) & (place < R)
        D, Y = torch.randn(n, ldd, device="cuda:0").to(T()[t]), torch.randn(R, ldy, device="cuda:0").to(T()[t])
        dY = torch.randn(R, lddy, device="cuda:0").to(T()[t])
        before = dY.clone()
        w = RNG(i).standard_normal((n, k)).astype(np.float32)
        dw = torch.full((n, k), NAN, device="cuda:0")
        g.combine_rows_grad(D, Y, dev(place.astype(np.int32)), dev(w), dY, dw, tokens=n, top=k, K=K, rows=R, dtype=t,
                            ldd=ldd, ldy=ldy, lddy=lddy)
        torch.cuda.synchronize()
        d, y, got = host(D)[:, :K], host(Y)[:, :K], host(dY)
        touched = np.zeros(R, dtype=bool)
        ref_dw, den = np.zeros((n, k)), np.zeros((n, k))
        for r in range(n):
            for j in range(k):
                if ok[r, j]:
                    ref = float(w[r, j]) * d[r]
                    # rounded to fp32 and then to the type
                    check(got[place[r, j], :K], ref, (HALF_STEP[t] * (1 + U32) + U32) * np.abs(ref), t, (n, k, K))
                    touched[place[r, j]] = True
                    ref_dw[r, j], den[r, j] = d[r] @ y[place[r, j]], np.abs(d[r]) @ np.abs(y[place[r, j]])
        check(host(dw), ref_dw, (K + 2) * U32 * den, "f32", (n, k, K))
        idle = torch.from_numpy(~touched).cuda()
        assert torch.equal(bits(dY[idle]), bits(before[idle])) and torch.equal(bits(dY[:, K:]), bits(before[:, K:]))


def test_combine_grad_against_differences(g):
    """combine is linear in the rows and in the weights: its differences are its gradients, exactly but
    for rounding."""
    import torch
    n, k, K = 9, 3, 40
    rng = RNG(6)
    place = rng.permutation(n * k).reshape(n, k)
    Y, D = dev(rng.standard_normal((n * k, K)), "f16"), dev(rng.standard_normal((n, K)), "f16")
    w = rng.standard_normal((n, k)).astype(np.float32)
    dY, dw = torch.zeros_like(Y), torch.zeros(n, k, device="cuda:0")
    g.combine_rows_grad(D, Y, dev(place.astype(np.int32)), dev(w), dY, dw, tokens=n, top=k, K=K, rows=n * k, dtype="f16")
    torch.cuda.synchronize()
    y, d = host(Y), host(D)

    def f(wv, yv):
        return sum((d[t] * (wv[t, j] * yv[place[t, j]])).sum() for t in range(n) for j in range(k))

    step_y, step_w = rng.standard_normal(y.shape), rng.standard_normal((n, k))
    w64 = w.astype(np.float64)
    diff = (f(w64, y + step_y) - f(w64, y - step_y)) / 2
    assert abs((host(dY) * step_y).sum() - diff) <= (HALF_STEP["f16"] + 2 * U32) * np.abs(host(dY) * step_y).sum() + 1e-9
    diff = (f(w64 + step_w, y) - f(w64 - step_w, y)) / 2
    lim = sum(np.abs(step_w[t, j]) * (np.abs(d[t]) @ np.abs(y[place[t, j]])) for t in range(n) for j in range(k))
    assert abs((host(dw) * step_w).sum() - diff) <= (K + 2) * U32 * lim + 1e-9


def test_rows_far_addresses(g):
    """Rows further than 2^32 bytes from the start."""
    import torch
    n, k, K, R, ld = 3, 2, 96, 140000, 16384
    A, X = torch.zeros(R, ld, device="cuda:0", dtype=torch.bfloat16), torch.randn(n, K, device="cuda:0").to(torch.bfloat16)
    place = np.array([[R - 1, 5], [R - 9, R - 2], [0, R - 3]], dtype=np.int32)
    g.dispatch_rows(X, dev(place), A, tokens=n, top=k, K=K, rows=R, lda=ld)
    C = torch.empty_like(X)
    g.combine_rows(A, dev(place), C, tokens=n, top=k, K=K, rows=R, ldy=ld)
    assert torch.equal(C, 2 * X)
    R = 600000                                             # rows of 8 KB: the last pass 2^32 bytes
    Q, S = torch.zeros(R * 8192, dtype=torch.uint8, device="cuda:0"), torch.zeros(R, 16, dtype=torch.uint8, device="cuda:0")
    q1, s1 = torch.zeros(n, K // 2, dtype=torch.uint8, device="cuda:0"), torch.zeros(n, 3, dtype=torch.uint8, device="cuda:0")
    place[:, 0] = [R - 1, R - 7, R - 4]
    g.quantize_mx(X, Q, S, M=n, K=K, place=dev(place), top=k, rows=R, ldq=2 ** 14, lds=16)
    g.quantize_mx(X, q1, s1, M=n, K=K)
    torch.cuda.synchronize()
    for t in range(n):
        r = int(place[t, 0])
        assert torch.equal(Q[r * 8192:r * 8192 + K // 2], q1[t]) and torch.equal(S[r, :3], s1[t])


@pytest.mark.parametrize("t,n,k,K,ld", [("bf16", 1601, 8, 2051, 2053), ("bf16", 8200, 8, 2056, 2056),
                                        ("f16", 30001, 1, 1001, 1002), ("f32", 4099, 3, 5600, 5600),
                                        ("f32", 16500, 2, 2052, 2053)])
def test_rows_past_the_caches(g, t, n, k, K, ld):
    """Rows of more than 48 and 256 MB, which take loads and stores that are not kept: dispatch exactly, the
    sums of at most 8 and K products in fp32 with one rounding."""
    import torch
    gen = torch.Generator(device="cuda:0").manual_seed(n)
    R = n * k
    place = torch.randperm(R, device="cuda:0", generator=gen).view(n, k)
    place[5] = -1
    X, Y, A, dY = (torch.randn(rows, ld, device="cuda:0", generator=gen).to(T()[t]) for rows in (n, R, R, R))
    C, w = torch.randn(n, ld, device="cuda:0", generator=gen).to(T()[t]), torch.rand(n, k, device="cuda:0", generator=gen)
    dw, before = torch.empty(n, k, device="cuda:0"), (A.clone(), C.clone(), dY.clone())
    p32, kw = place.int(), dict(tokens=n, top=k, K=K, rows=R, dtype=t)
    g.dispatch_rows(X, p32, A, ldx=ld, lda=ld, **kw)
    g.combine_rows(Y, p32, C, weight=w, beta=0.5, ldy=ld, ldc=ld, **kw)
    g.combine_rows_grad(X, Y, p32, w, dY, dw, ldd=ld, ldy=ld, lddy=ld, **kw)
    torch.cuda.synchronize()
    live = place >= 0
    at, tok = place[live], torch.arange(n, device="cuda:0")[:, None].expand(n, k)[live]
    want = before[0].clone()
    want[at, :K] = X[tok, :K]
    assert torch.equal(bits(A), bits(want))
    # a product, rounded to fp32 (or, where the compiler joins the product and the conversion, not) and then
    # to the type: within half a step of the type plus one of fp32 of the exact product, and of a subnormal
    # result within half the type's smallest number
    exact = w[live][:, None].double() * X[tok, :K].double()
    off = (dY[at, :K].double() - exact).abs()
    assert (off <= (HALF_STEP[t] + 1.01 * U32) * exact.abs() + TINY[t]).all()
    dY[at, :K] = before[2][at, :K]
    assert torch.equal(bits(dY), bits(before[2]))
    assert torch.equal(bits(C[:, K:]), bits(before[1][:, K:])) and (dw[5] == 0).all()
    x, h = X[:, :K].double(), HALF_STEP[t]
    ref, den = 0.5 * before[1][:, :K].double(), 0.5 * before[1][:, :K].double().abs()
    for j in range(k):
        y = torch.where(live[:, j, None], Y[place[:, j].clamp_min(0), :K].double(), 0.0)
        ref += w[:, j, None].double() * y
        den += w[:, j, None].double() * y.abs()
        dot, size = (x * y).sum(dim=1), (x * y).abs().sum(dim=1)
        assert ((dw[:, j].double() - dot).abs() <= (K + 2) * U32 * size).all()
    # (fp16's subnormal numbers lie 2^-24 apart: half of that, TINY, is the least that a rounding is off by)
    lim = (k + 1) * U32 * den + h * (ref.abs() + (k + 1) * U32 * den) + TINY[t]
    assert ((C[:, :K].double() - ref).abs() <= lim).all()


# ---------------------------------------------------------------------------- quantize_mx --

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])      # ties: to the even code


def mx_reference(x):
    """Codes (0 .. 15) and scale bytes of rows x in 64 bits."""
    n, K = x.shape
    v = x.reshape(n, K // 32, 32)
    big = np.abs(v).max(axis=2)
    bad = ~np.isfinite(v).all(axis=2)
    e = np.where(big > 0, np.frexp(np.where(bad, 1.0, big))[1] - 3, -127).clip(-127, 127)
    e[big == 0] = -127
    y = np.abs(np.ldexp(np.where(bad[:, :, None], 0.0, v), -e[:, :, None]))
    code = np.zeros(v.shape, dtype=np.int64)
    for i, b in enumerate(BORDERS):
        code += (y >= b) if i % 2 else (y > b)
    code |= np.signbit(v).astype(np.int64) << 3
    code[bad] = 0
    return code.reshape(n, K), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1).astype(np.int64)


def values(code, s):
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    with np.errstate(invalid="ignore"):
        sc = np.where(s == 255, NAN, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v.reshape(*s.shape, 32) * sc[:, :, None]).reshape(code.shape)


def quant(g, X, K, t, pad=0):
    """Codes and scale bytes of the first K columns of a device matrix."""
    import torch
    n, ldx = X.shape
    Q = torch.full((n, K // 2 + pad), 0xAB, dtype=torch.uint8, device="cuda:0")
    S = torch.full((n, K // 32 + pad), 0xAB, dtype=torch.uint8, device="cuda:0")
    g.quantize_mx(X, Q, S, M=n, K=K, x_type=t, ldx=ldx, ldq=K + 2 * pad, lds=K // 32 + pad)
    torch.cuda.synchronize()
    assert (Q[:, K // 2:] == 0xAB).all() and (S[:, K // 32:] == 0xAB).all()
    return unpack(Q[:, :K // 2].cpu().numpy()), S[:, :K // 32].cpu().numpy()


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_quantize_every_16_bit_value(g, t):
    """All 65536 values: next to values of their own size, and next to every power of two above them."""
    import torch
    every = torch.arange(65536, dtype=torch.int32, device="cuda:0").to(torch.int16).view(T()[t])
    X = every.view(256, 256)
    code, s = quant(g, X, 256, t)
    rc, rs = mx_reference(host(X))
    assert np.array_equal(s, rs) and np.array_equal(code, rc)
    finite = every[torch.isfinite(every)]
    for up in (1, 2, 4, 8, 16):
        # blocks of 31 values and their largest's multiple
        v = finite[:finite.numel() // 31 * 31].view(-1, 31)
        big = (v.float().abs().amax(dim=1, keepdim=True) * up).clamp_max(torch.finfo(v.dtype).max).to(v.dtype)
        X = torch.cat([v, big], dim=1)
        code, s = quant(g, X, 32, t)
        rc, rs = mx_reference(host(X))
        assert np.array_equal(s, rs) and np.array_equal(code, rc), up


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantize_sizes(g, t):
    import torch
    for i, (n, K) in enumerate([(1, 32), (1, 4096), (3, 64), (17, 96), (5, 2048), (4, 2080), (2, 4128), (300, 512), (2, 40000 // 32 * 32)]):
        print(f"[quantize_mx] {t} {n} {K}", flush=True)
        gen = torch.Generator(device="cuda:0").manual_seed(i)
        X = torch.randn(n, K + i % 3, device="cuda:0", generator=gen)
        X *= torch.exp2(torch.randint(-12, 12, X.shape, device="cuda:0", generator=gen).float())
        X = X.to(T()[t])
        X[0, :32] = 0
        if K > 64:
            X[0, 33] = INF
            X[n - 1, 64] = NAN
        code, s = quant(g, X, K, t, pad=i % 2)
        rc, rs = mx_reference(host(X)[:, :K])
        assert np.array_equal(s, rs) and np.array_equal(code, rc), (n, K)


def test_quantize_fp32_extremes(g):
    """Subnormal numbers, the largest ones, both ends of the scales, and values at the borders."""
    import torch
    rng = RNG(2)
    e = np.concatenate([np.arange(-149, 128), [127] * 3])
    x = np.ldexp(1 + rng.random((e.size, 32)), e[:, None]).astype(np.float32)
    x *= rng.choice([-1, 1], x.shape)
    x[:, 1:8] = np.ldexp(BORDERS, e[:, None].clip(-140, 125) - 2)      # ties where the block's largest is 1 .. 2 times 2^e
    x[:, 8] = 0.0
    x[:, 9] = -0.0
    X = dev(x.astype(np.float32))
    code, s = quant(g, X, 32, "f32")
    rc, rs = mx_reference(host(X))
    assert np.array_equal(s, rs) and np.array_equal(code, rc)


def test_quantize_to_places(g):
    import torch
    for n, k, K in ((1, 1, 32), (16, 2, 2048), (33, 4, 2080), (7, 8, 160)):
        R = n * k + 5
        place = places(n, k, R, 3)
        X = torch.randn(n, K, device="cuda:0").to(torch.bfloat16)
        Q, S = (torch.full((R, w), 0xCD, dtype=torch.uint8, device="cuda:0") for w in (K // 2, K // 32))
        g.quantize_mx(X, Q, S, M=n, K=K, place=dev(place.astype(np.int32)), top=k, rows=R)
        q1, s1 = (torch.zeros(n, w, dtype=torch.uint8, device="cuda:0") for w in (K // 2, K // 32))
        g.quantize_mx(X, q1, s1, M=n, K=K)
        want_q, want_s = torch.full_like(Q, 0xCD), torch.full_like(S, 0xCD)
        for r in range(n):
            for j in range(k):
                if 0 <= place[r, j] < R:
                    want_q[place[r, j]], want_s[place[r, j]] = q1[r], s1[r]
        torch.cuda.synchronize()
        assert torch.equal(Q, want_q) and torch.equal(S, want_s)


# ----------------------------------------------------------------------- grouped products --

STREAM, TILES = 5, [2, 3, 4]
MANY = [0, 3, 1, 0, 17] * 14 + [33]  # 71 groups: more than a wave has lanes
SIZES = [[0], [1], [5, 0, 7], [0, 0, 3, 0], [64, 65, 1, 0, 127], [300, 2, 513], MANY]
DIMS = [(1, 32), (33, 64), (64, 256), (100, 96), (264, 544), (136, 2080), (40, 1024)]


def effective(offsets, M):
    return np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, M))


def random_mx(rng, n, K, ld, lds, spread=4):
    """Packed rows of leading dimension ld (elements) and scale rows, garbage past K; their values."""
    code = rng.integers(0, 16, (n, ld))
    q = (code[:, ::2] | code[:, 1::2] << 4).astype(np.uint8)
    s = np.full((n, lds), 255, dtype=np.uint8)
    s[:, :K // 32] = rng.integers(127 - spread, 128 + spread, (n, K // 32))
    return q, s, values(code[:, :K], s[:, :K // 32])


def gelu(x):
    with np.errstate(invalid="ignore"):
        return 0.5 * x * erfc(-x / np.sqrt(2.0))


def run_mx(g, sizes, N, K, *, ct="bf16", kernel=0, alpha=1.0, beta=0.0, bias=False, do_gelu=False, lda=None, ldb=None,
           ldc=None, ldsa=None, ldsb=None, gap=0, shared=False, offsets=None, M=None, seed=0, shift=0, stream=None,
           no_offsets=False):
    """One call against the plain form.  shift: bytes that the operands start after a multiple of 16."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    G = len(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64) if offsets is None else np.asarray(offsets, dtype=np.int64)
    M = int(off[-1]) if M is None else M
    eff = effective(off, M)
    rng = RNG([seed, N, K])
    kb = (K // 32 + 15) // 16 * 16
    lda, ldb, ldc, ldsa, ldsb = lda or (K + 31) // 32 * 32, ldb or (K + 31) // 32 * 32, ldc or N, ldsa or kb, ldsb or kb
    qa, sa, a = random_mx(rng, M, K, lda, ldsa)
    inside = np.zeros(M, dtype=bool)
    for q in range(G):
        inside[eff[q]:eff[q + 1]] = True
    sa[~inside] = 255
    H = 1 if shared else G
    qb, sb, b = [], [], []
    for q in range(H):
        x, y, z = random_mx(rng, N, K, ldb, ldsb)
        qb += [x.ravel(), np.full(gap, 0x77, dtype=np.uint8)]
        sb += [y.ravel(), np.full(gap, 255, dtype=np.uint8)]
        b.append(z)

    def put(x):
        t = torch.zeros(x.size + 64, dtype=torch.uint8, device="cuda:0")
        t[shift:shift + x.size] = torch.from_numpy(np.ascontiguousarray(x).ravel()).cuda()
        return t[shift:]

    A, SA, B, SB = put(qa), put(sa), put(np.concatenate(qb)), put(np.concatenate(sb))
    C = dev(rng.standard_normal((M, ldc)), ct)
    before = C.clone()
    bias_h = rng.standard_normal((G, N)).astype(np.float32) if bias else None
    db = dev(bias_h) if bias else None
    g.run_grouped_mx(A, SA, B, SB, C, None if no_offsets else dev(off), groups=G, M=M, N=N, K=K, c_type=ct, alpha=alpha,
                     beta=beta, epilogue=(tmm.GEMM_EPI_BIAS if bias else 0) | (tmm.GEMM_EPI_GELU if do_gelu else 0),
                     bias=db, lda=lda, ldsa=ldsa, ldb=ldb, ldsb=ldsb,
                     stride_b=0 if shared else N * ldb + 2 * gap, stride_sb=0 if shared else N * ldsb + gap, ldc=ldc,
                     kernel=kernel, stream=stream)
    torch.cuda.synchronize()
    cin, got = host(before), host(C)
    ref, D = cin[:, :N].copy(), np.zeros((M, N))
    for q in range(G):
        r = slice(eff[q], eff[q + 1])
        w = b[0 if shared else q]
        v, d = alpha * (a[r] @ w.T), abs(alpha) * (np.abs(a[r]) @ np.abs(w).T)
        if beta:
            v, d = v + beta * cin[r, :N], d + np.abs(beta * cin[r, :N])
        if bias:
            v, d = v + bias_h[q].astype(np.float64), d + np.abs(bias_h[q])
        ref[r], D[r] = gelu(v) if do_gelu else v, d
    tol = K * 2.0 ** -23 + HALF_STEP[ct] + (20 if do_gelu else 4) * U32
    check(got[inside][:, :N], ref[inside], tol * np.maximum(D, np.abs(ref))[inside], ct, (sizes[:6], N, K, ct, kernel))
    out = torch.from_numpy(~inside).cuda()
    assert torch.equal(bits(C[out]), bits(before[out])), "rows of no group"
    assert torch.equal(bits(C[:, N:]), bits(before[:, N:])), "columns past N"
    return C


@pytest.mark.parametrize("kernel", [STREAM, 0])
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_mx_sizes(g, ct, kernel):
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(DIMS):
            print(f"[mx] {ct} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_mx(g, sizes, N, K, ct=ct, kernel=kernel, seed=10 * i + j, bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                   alpha=0.75 if j % 2 else 1.0, beta=-0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", TILES)
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_mx_tiles(g, ct, kernel):
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(DIMS):
            N = -(-N // 4) * 4
            print(f"[mx] {ct} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_mx(g, sizes, N, K, ct=ct, kernel=kernel, seed=10 * i + j, bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                   alpha=0.75 if j % 2 else 1.0, beta=-0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", [0, STREAM] + TILES)
def test_mx_strides_and_rows_of_no_group(g, kernel):
    run_mx(g, [40, 0, 90], 72, 416, ct="bf16", kernel=kernel, lda=448, ldb=512, ldc=80, ldsa=32, ldsb=48, gap=16,
           offsets=[7, 47, 47, 137], M=150, bias=True, seed=3)
    run_mx(g, [40, 9, 90], 72, 416, ct="f16", kernel=kernel, shared=True, seed=4)
    for offsets in ([0, 50, 20, 100], [-5, 30, 300, 80], [90, 10, 20, 30], [2 ** 40, 0, 5, 9], [-2 ** 62, 2 ** 62, 3, 2 ** 62]):
        run_mx(g, [0, 0, 0], 64, 64, kernel=kernel, offsets=offsets, M=100, seed=5)
    run_mx(g, [70], 40, 96, kernel=kernel, no_offsets=True, seed=6)


def test_mx_any_alignment(g):
    """Operands and scales that start and lie anywhere go through the streaming kernel."""
    for shift in (1, 3, 8):
        for sizes in ([1], [17, 0, 40], [150, 200]):
            run_mx(g, sizes, 37, 544, kernel=0, lda=546, ldb=550, ldc=39, ldsa=17, ldsb=19, gap=5, shift=shift, seed=shift)


def test_mx_one_token_and_wide(g):
    for M in (1, 2, 15, 16, 17, 31, 33):
        run_mx(g, [M], 1000, 8192, no_offsets=True, seed=M, bias=True)
    run_mx(g, [700], 2000, 2048, no_offsets=True, do_gelu=True, bias=True)


def test_mx_k_of_zero(g):
    import torch
    import tiled_matrix_multiply_amd as tmm
    C = torch.full((20, 8), 3.0, device="cuda:0", dtype=torch.bfloat16)
    bias = torch.arange(8, device="cuda:0").float()
    g.run_grouped_mx(None, None, None, None, C, None, groups=1, M=20, N=8, K=0, beta=0.5, bias=bias,
                     epilogue=tmm.GEMM_EPI_BIAS)
    assert torch.equal(C.float(), (1.5 + bias).expand(20, 8))


@pytest.mark.parametrize("kernel", [STREAM] + TILES)
def test_mx_nan_scales_stay_in_their_rows(g, kernel):
    import torch
    rng = RNG(1)
    qa, sa, _ = random_mx(rng, 96, 512, 512, 16)
    qb, sb, _ = random_mx(rng, 64, 512, 512, 16)
    sa[10, 3], sa[70, 15], sb[5, 0] = 255, 255, 255
    qa[10, 48:64] = 0                                   # codes 0, as quantize_mx writes them
    C = torch.zeros(96, 64, device="cuda:0", dtype=torch.bfloat16)
    g.run_grouped_mx(dev(qa), dev(sa), dev(qb), dev(sb), C, None, groups=1, M=96, N=64, K=512, ldsa=16, ldsb=16, kernel=kernel)
    bad = torch.isnan(C).cpu()
    want = torch.zeros(96, 64, dtype=torch.bool)
    want[10], want[70], want[:, 5] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("kernel", [STREAM] + TILES)
def test_mx_far_addresses(g, kernel):
    """Rows of A, their results and a group's matrix further than 2^32 bytes from the start."""
    import torch
    M, N, K, ld, ldc = 530, 40, 64, 2 ** 24, 2 ** 23
    rng = RNG([kernel, 77])
    qa, sa, a = random_mx(rng, M, K, K, 16)
    qb, sb, b = random_mx(rng, 2 * N, K, K, 16)
    A = torch.zeros(M, ld // 2, dtype=torch.uint8, device="cuda:0")         # 4.4 GB
    A[:, :K // 2] = torch.from_numpy(qa).cuda()
    far = 2 ** 32 + 4096
    B = torch.zeros(far + N * K, dtype=torch.uint8, device="cuda:0")
    for i in range(2):
        B[i * far:i * far + N * K // 2] = torch.from_numpy(qb[i * N:(i + 1) * N].ravel()).cuda()
    C = torch.zeros(M, ldc, dtype=torch.bfloat16, device="cuda:0")           # 8.9 GB
    off = dev(np.array([0, 3, M], dtype=np.int64))
    SA, SB = torch.from_numpy(sa).cuda(), torch.from_numpy(sb).cuda()
    g.run_grouped_mx(A, SA, B, SB, C, off, groups=2, M=M, N=N, K=K, lda=ld, ldsa=16, ldsb=16, stride_b=2 * far,
                     stride_sb=16 * N, ldc=ldc, kernel=kernel)
    torch.cuda.synchronize()
    w = [b[:N], b[N:]]
    ref = np.concatenate([a[:3] @ w[0].T, a[3:] @ w[1].T])
    D = np.concatenate([np.abs(a[:3]) @ np.abs(w[0]).T, np.abs(a[3:]) @ np.abs(w[1]).T])
    check(host(C[:, :N].contiguous()), ref, (K * 2.0 ** -23 + HALF_STEP["bf16"] + 4 * U32) * D, "bf16", kernel)
    assert not C[:, N:N + 64].any() and not C[:, ldc - 64:].any()


def test_mx_refuses_what_a_kernel_cannot(g):
    import torch
    import tiled_matrix_multiply_amd as tmm
    z = torch.zeros(4096, dtype=torch.uint8, device="cuda:0")
    C = torch.zeros(16, 16, device="cuda:0", dtype=torch.bfloat16)
    for kernel, shift in ((1, 0), (2, 1), (3, 1), (4, 1), (6, 0), (-1, 0)):
        with pytest.raises(tmm.GemmError):
            g.run_grouped_mx(z[shift:], z[768:], z[1536:], z[2304:], C, None, groups=1, M=16, N=16, K=64, ldsa=16,
                             ldsb=16, kernel=kernel)
    # scale rows that are no multiple of 16 bytes: tiles refuse, AUTO streams
    with pytest.raises(tmm.GemmError):
        g.run_grouped_mx(z, z[768:], z[1536:], z[2304:], C, None, groups=1, M=16, N=16, K=64, kernel=2)
    g.run_grouped_mx(z, z[768:], z[1536:], z[2304:], C, None, groups=1, M=16, N=16, K=64)


# ---------------------------------------------------------------------------- together --

def layer(g, x, logits_, w1, s1, w2, s2, b1, k, ws, bufs, stream=None):
    """A mixture-of-experts perceptron in MXFP4, as a program would call it."""
    import tiled_matrix_multiply_amd as tmm
    n, K = x.shape
    E, Hd = w1.shape[0], w1.shape[1]
    R = n * k
    g.route(logits_, bufs["expert"], bufs["weight"], bufs["place"], bufs["offsets"], tokens=n, experts=E, top=k,
            score="softmax", renorm=True, workspace=ws, stream=stream)
    g.quantize_mx(x, bufs["qa"], bufs["sa"], M=n, K=K, place=bufs["place"], top=k, rows=R, lds=bufs["sa"].shape[1],
                  stream=stream)
    g.run_grouped_mx(bufs["qa"], bufs["sa"], w1, s1, bufs["h"], bufs["offsets"], groups=E, M=R, N=Hd, K=K,
                     ldsa=bufs["sa"].shape[1], ldsb=s1.shape[2], epilogue=tmm.GEMM_EPI_BIAS | tmm.GEMM_EPI_GELU, bias=b1,
                     stream=stream)
    g.quantize_mx(bufs["h"], bufs["qh"], bufs["sh"], M=R, K=Hd, lds=bufs["sh"].shape[1], stream=stream)
    g.run_grouped_mx(bufs["qh"], bufs["sh"], w2, s2, bufs["y"], bufs["offsets"], groups=E, M=R, N=K, K=Hd,
                     ldsa=bufs["sh"].shape[1], ldsb=s2.shape[2], stream=stream)
    g.combine_rows(bufs["y"], bufs["place"], bufs["out"], tokens=n, top=k, K=K, rows=R, weight=bufs["weight"],
                   stream=stream)


def make_layer(g, n, E, k, K, Hd, seed=0):
    import torch
    import tiled_matrix_multiply_amd as tmm
    gen = torch.Generator(device="cuda:0").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda:0", generator=gen)

    def zeros(*shape, dtype=torch.uint8):
        return torch.zeros(*shape, dtype=dtype, device="cuda:0")

    up = lambda v: (v + 15) // 16 * 16
    x, lg = normal(n, K).to(torch.bfloat16), normal(n, E)
    lg[n - 1] = -INF                                    # a padded token
    w1f, w2f = (normal(E, Hd, K) * K ** -0.5).to(torch.bfloat16), (normal(E, K, Hd) * Hd ** -0.5).to(torch.bfloat16)
    w1, s1, w2, s2 = zeros(E, Hd, K // 2), zeros(E, Hd, up(K // 32)), zeros(E, K, Hd // 2), zeros(E, K, up(Hd // 32))
    g.quantize_mx(w1f, w1, s1, M=E * Hd, K=K, lds=s1.shape[2])
    g.quantize_mx(w2f, w2, s2, M=E * K, K=Hd, lds=s2.shape[2])
    R = n * k
    bufs = {"expert": zeros(n, k, dtype=torch.int32), "weight": zeros(n, k, dtype=torch.float32),
            "place": zeros(n, k, dtype=torch.int32), "offsets": zeros(E + 1, dtype=torch.int64),
            "qa": zeros(R, K // 2), "sa": zeros(R, up(K // 32)), "h": zeros(R, Hd, dtype=torch.bfloat16),
            "qh": zeros(R, Hd // 2), "sh": zeros(R, up(Hd // 32)), "y": zeros(R, K, dtype=torch.bfloat16),
            "out": zeros(n, K, dtype=torch.bfloat16)}
    ws = zeros(max(16, tmm.route_workspace_bytes(n, E)))
    return (x, lg, w1, s1, w2, s2, 0.1 * normal(E, Hd), k, ws, bufs)


@pytest.mark.parametrize("n", [1, 50, 700])
def test_layer_in_mxfp4(g, n):
    """Route, quantize to the experts, two products, combine: each step against 64 bits from the bits
    that went into it."""
    import torch
    E, k, K, Hd = 12, 3, 256, 384
    args = make_layer(g, n, E, k, K, Hd)
    x, lg, w1, s1, w2, s2, b1, _, _, bufs = args
    layer(g, *args)
    torch.cuda.synchronize()
    expert, weight, place, off = reference(host(lg), k, "softmax", None, 1, 1, 1, True, 1.0)
    assert np.array_equal(bufs["expert"].cpu().numpy(), expert) and np.array_equal(bufs["place"].cpu().numpy(), place)
    assert np.array_equal(bufs["offsets"].cpu().numpy(), off)
    dec = lambda q, s, k_: values(unpack(q.cpu().numpy()), s[:, :k_ // 32].cpu().numpy())
    code, s = mx_reference(host(x))
    a = values(code, s)
    h, y = host(bufs["h"]), host(bufs["y"])
    qh = dec(bufs["qh"], bufs["sh"], Hd)
    assert np.array_equal(qh[:off[-1]], values(*mx_reference(h[:off[-1]])))
    rows = np.zeros((n * k, K))
    for t in range(n):
        for j in range(k):
            if place[t, j] >= 0:
                rows[place[t, j]] = a[t]
    for e in range(E):
        r = slice(off[e], off[e + 1])
        m1, m2 = dec(w1[e], s1[e], K), dec(w2[e], s2[e], Hd)
        bias = host(b1[e])
        v, d = rows[r] @ m1.T + bias, np.abs(rows[r]) @ np.abs(m1).T + np.abs(bias)
        ref = gelu(v)
        check(h[r], ref, (K * 2.0 ** -23 + HALF_STEP["bf16"] + 20 * U32) * np.maximum(d, np.abs(ref)), "bf16", ("h", e))
        v, d = qh[r] @ m2.T, np.abs(qh[r]) @ np.abs(m2).T
        check(y[r], v, (Hd * 2.0 ** -23 + HALF_STEP["bf16"] + 4 * U32) * np.maximum(d, np.abs(v)), "bf16", ("y", e))
    ok = place >= 0
    w = host(bufs["weight"])
    yy = np.where(ok[:, :, None], y[np.where(ok, place, 0)], 0.0)
    ref, den = (w[:, :, None] * yy).sum(axis=1), (np.abs(w)[:, :, None] * np.abs(yy)).sum(axis=1)
    check(host(bufs["out"]), ref, 5 * U32 * den + HALF_STEP["bf16"] * (np.abs(ref) + 5 * U32 * den), "bf16", "out")
    assert (host(bufs["out"])[n - 1] == 0).all()       # the padded token


@pytest.mark.parametrize("n", [4, 300])
def test_layer_in_a_graph(g, n):
    """Captured and replayed with other tokens, with eager work between the replays; every replay equals
    the eager result."""
    import torch
    args = make_layer(g, n, 16, 2, 128, 256, seed=1)
    x, lg, bufs = args[0], args[1], args[-1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(g, *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(g, *args)
    other = make_layer(g, n, 16, 2, 128, 256, seed=1)
    for i in range(4):
        gen = torch.Generator(device="cuda:0").manual_seed(50 + i)
        x.copy_(torch.randn(x.shape, device="cuda:0", generator=gen))
        lg.copy_(torch.randn(lg.shape, device="cuda:0", generator=gen))
        other[0].copy_(x)
        other[1].copy_(lg)
        layer(g, *other)
        for b in bufs.values():
            b.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("expert", "weight", "place", "offsets", "out"):
            assert torch.equal(bufs[name], other[-1][name]), (i, name)


@pytest.mark.parametrize("n", [3, 130])
def test_training_step_in_a_graph(g, n):
    """The router and the rows' ways there and back with all their gradients, captured, and replayed with
    other tokens and eager work between: every replay equals the eager result."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    E, k, K = 12, 3, 520
    R = n * k
    ws = torch.zeros(max(16, tmm.route_workspace_bytes(n, E)), dtype=torch.uint8, device="cuda:0")

    def make():
        i32 = [torch.empty(n, k, dtype=torch.int32, device="cuda:0") for _ in range(2)]
        f32 = [torch.empty(n, k, device="cuda:0") for _ in range(2)]
        rows = [torch.zeros(R, K, device="cuda:0", dtype=torch.bfloat16) for _ in range(2)]
        return dict(x=torch.zeros(n, K, device="cuda:0", dtype=torch.bfloat16), lg=torch.zeros(n, E, device="cuda:0"),
                    d=torch.zeros(n, K, device="cuda:0", dtype=torch.bfloat16), expert=i32[0], place=i32[1], w=f32[0],
                    dw=f32[1], a=rows[0], dy=rows[1], off=torch.empty(E + 1, dtype=torch.int64, device="cuda:0"),
                    out=torch.empty(n, K, device="cuda:0", dtype=torch.bfloat16),
                    dx=torch.empty(n, K, device="cuda:0", dtype=torch.bfloat16), dl=torch.empty(n, E, device="cuda:0"))

    def step(b):
        kw = dict(tokens=n, top=k, K=K, rows=R)
        g.route(b["lg"], b["expert"], b["w"], b["place"], b["off"], tokens=n, experts=E, top=k, workspace=ws)
        g.dispatch_rows(b["x"], b["place"], b["a"], **kw)
        g.combine_rows(b["a"], b["place"], b["out"], weight=b["w"], **kw)
        g.combine_rows_grad(b["d"], b["a"], b["place"], b["w"], b["dy"], b["dw"], **kw)
        g.combine_rows(b["dy"], b["place"], b["dx"], **kw)
        g.route_grad(b["lg"], b["expert"], b["dw"], b["dl"], tokens=n, experts=E, top=k)

    b, eager = make(), make()
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(4):
        gen = torch.Generator(device="cuda:0").manual_seed(i)
        for name in ("x", "lg", "d"):
            b[name].copy_(torch.randn(b[name].shape, device="cuda:0", generator=gen))
            eager[name].copy_(b[name])
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in b:
            assert torch.equal(b[name], eager[name]), (i, name)


def test_two_streams_at_once(g):
    """Two layers with workspaces of their own on two streams, and the same again alone: the same bits."""
    import torch
    made = [make_layer(g, 400, 32, 4, 256, 256, seed=s) for s in (2, 3)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(3):
        for a, s in zip(made, streams):
            with torch.cuda.stream(s):
                layer(g, *a)
    torch.cuda.synchronize()
    for a in made:
        got = {k: v.clone() for k, v in a[-1].items()}
        for v in a[-1].values():
            v.zero_()
        layer(g, *a)
        torch.cuda.synchronize()
        for k in ("expert", "weight", "place", "offsets", "out"):
            assert torch.equal(got[k], a[-1][k]), k


def test_training_step_of_the_rows(g):
    """dispatch, a product for each expert, combine, and all gradients back to the logits, against
    autograd of the plain form in 64 bits."""
    import torch
    n, E, k, K = 60, 6, 2, 48
    rng = RNG(5)
    x, lg = dev(rng.standard_normal((n, K)), "f32"), dev(rng.standard_normal((n, E)), "f32")
    expert, place = (torch.empty(n, k, dtype=torch.int32, device="cuda:0") for _ in range(2))
    weight, off = torch.empty(n, k, device="cuda:0"), torch.empty(E + 1, dtype=torch.int64, device="cuda:0")
    g.route(lg, expert, weight, place, off, tokens=n, experts=E, top=k)
    R = n * k
    a, dy, y, da = (torch.zeros(R, K, device="cuda:0") for _ in range(4))
    out, dx = torch.empty(n, K, device="cuda:0"), torch.empty(n, K, device="cuda:0")
    dw, dl = torch.empty(n, k, device="cuda:0"), torch.empty(n, E, device="cuda:0")
    kw = dict(tokens=n, top=k, K=K, rows=R, dtype="f32")
    g.dispatch_rows(x, place, a, **kw)
    scale = torch.repeat_interleave(torch.arange(1.0, E + 1, device="cuda:0"), off.diff())   # expert e: times e + 1
    torch.mul(a, scale[:, None], out=y)
    g.combine_rows(y, place, out, weight=weight, **kw)
    d = dev(rng.standard_normal((n, K)), "f32")
    g.combine_rows_grad(d, y, place, weight, dy, dw, **kw)
    torch.mul(dy, scale[:, None], out=da)
    g.combine_rows(da, place, dx, **kw)
    g.route_grad(lg, expert, dw, dl, tokens=n, experts=E, top=k)
    torch.cuda.synchronize()
    xr, lr = x.double().cpu().requires_grad_(), lg.double().cpu().requires_grad_()
    p = torch.softmax(lr, dim=1).gather(1, expert.cpu().long())
    ref = (p[:, :, None] * (expert.cpu().double() + 1)[:, :, None] * xr[:, None, :]).sum(dim=1)
    ref.backward(d.double().cpu())
    # every quantity is a sum of at most 48 + 2 products of numbers within fp32 roundings of the reference's
    for got, want in ((out, ref.detach()), (dx, xr.grad), (dl, lr.grad)):
        assert (got.double().cpu() - want).norm() <= 100 * U32 * want.norm()
