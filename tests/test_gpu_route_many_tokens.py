"""The router between a thousand tokens and seventy thousand, where workgroups hold 16, 32 or 64 of them, on both
sides of each border; a table of counts longer than one pass over it; and runs of experts that do not fit the
lanes.  Choices, places and offsets have to be equal, the weights' bounds are test_gpu_experts.py's."""
import numpy as np
import pytest

from test_gpu_experts import INF, RNG, check_route, dev, g, logits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,kw", [
    (256, 8, dict(kind="sigmoid", groups=8, best=4, of=2, renorm=True, scale=2.5)),   # two passes of a wave from 64 tokens on
    (256, 16, dict(kind="softmax")),
    (8, 2, dict(kind="softmax", renorm=True)),
    (60, 4, dict(kind="softmax", renorm=True)),
    (300, 5, dict(kind="sigmoid", groups=4, best=2)),
    (600, 20, dict(kind="softmax")),
])
def test_route_tokens_to_a_workgroup(g, E, k, kw):  # noqa: F811
    for n in (1039, 4095, 4096, 4097, 8191, 8192, 8193, 12000):
        if n * E > 2500000:
            continue
        print(f"[route] many tokens {E} {k} {n}", flush=True)
        x = logits(n, E, k)
        x[n - 40:] = -INF                                   # padding
        x[n // 3, 1:] = -INF
        bias = 0.2 * RNG([E, k]).standard_normal(E) if kw["kind"] == "sigmoid" else None
        check_route(g, x, k, "bf16" if n % 2 else "f32", bias=bias, **kw)


def plan(expert, E):
    """Places and offsets of given choices, by a stable sort."""
    import torch
    flat = expert.long().flatten()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    return torch.where(flat < 0, -1, place).view(expert.shape), torch.cat([counts.new_zeros(1), counts.cumsum(0)])


# (tokens, experts): a thread of the second kernel adds up 1000 rows of counts at a time, 4 threads to a column of
# 513 to 1024 experts and 16 of 129 to 256: more than 4000 blocks of 64 tokens, 8000 and 16000
@pytest.mark.parametrize("n,E,k", [(256001, 600, 1), (256064, 520, 2), (512100, 513, 1), (300000, 16, 3), (1100000, 256, 1)])
def test_route_long_tables(g, n, E, k):  # noqa: F811
    """Nearly all tokens to one expert, so that whole blocks count 64 there."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    gen = torch.Generator(device="cuda:0").manual_seed(n)
    x = torch.randn(n, E, device="cuda:0", generator=gen, dtype=torch.bfloat16)
    x[:, E // 2] += 6.0
    x[n - 1000:n - 3] = -INF
    expert, place = (torch.full((n, k), 7, dtype=torch.int32, device="cuda:0") for _ in range(2))
    weight, offsets = torch.empty(n, k, device="cuda:0"), torch.empty(E + 1, dtype=torch.int64, device="cuda:0")
    ws = torch.full((tmm.route_workspace_bytes(n, E),), 255, dtype=torch.uint8, device="cuda:0")
    print(f"[route] long table {n} {E} {k}", flush=True)
    g.route(x, expert, weight, place, offsets, tokens=n, experts=E, top=k, x_type="bf16", workspace=ws)
    torch.cuda.synchronize()
    # the choice: bf16 logits as numbers, equal ones in the experts' order (a stable sort of an order-keeping code)
    code = x.float().view(torch.int32).long()
    code = torch.where(code < 0, -(code & 0x7fffffff), code)
    left = code * 1024 + (1023 - torch.arange(E, device="cuda:0"))
    for j in range(k):
        best = left.amax(dim=1)
        e = (1023 - best % 1024).int()
        e[n - 1000:n - 3] = -1
        assert torch.equal(expert[:, j], e), j
        left.scatter_(1, e.clamp_min(0).long()[:, None], -2 ** 62)
    del left, code
    want_place, want_offsets = plan(expert, E)
    assert torch.equal(offsets, want_offsets) and torch.equal(place.long(), want_place)
    assert int(offsets.diff().max()) > n // 2


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_runs_that_do_not_fit_the_lanes(g, kind):  # noqa: F811
    """33 runs of 31 experts (and others) would need more than 64 lanes of 16: chosen in 64 bits throughout."""
    for E, groups, best, k in ((1023, 33, 5, 8), (1020, 60, 7, 32), (903, 43, 3, 4)):
        for n in (1, 20, 300):
            for of in (1, 2):
                for b in (False, True):
                    print(f"[route] runs {kind} {E} {groups} {n} {of} {b}", flush=True)
                    x = logits(n, E, k)
                    x[0, : E // 2] = -INF
                    if n > 2:
                        x[1] = -INF
                        x[2, 40:] = -INF
                    bias = 0.3 * RNG(E).standard_normal(E) if b else None
                    check_route(g, x, k, "f32", kind=kind, bias=bias, groups=groups, best=best, of=of, renorm=True)
