"""More groups than a wave has lanes, at the borders of its blocks of 64, with offsets that fall, leave
the matrix or stand still over whole blocks: inputs, references and tolerances of test_gpu_grouped.py."""
import numpy as np
import pytest

from test_gpu_grouped import g, run_grouped, run_i8, run_wgrad  # noqa: F401

pytestmark = pytest.mark.gpu

M = 300


def offsets(kind, groups):
    rng = np.random.default_rng(groups)
    if kind == "even":
        return np.arange(groups + 1) * M // groups
    if kind == "idle blocks":  # the rows belong to the last group of a block and to the very last one
        o = np.zeros(groups + 1, dtype=np.int64)
        o[64:] = 100
        o[groups] = M
        return o
    if kind == "falling":
        return np.arange(groups, -1, -1) * M // groups
    o = rng.integers(-50, M + 50, groups + 1)  # any
    o[groups // 2] = 2 ** 40
    return o if kind == "any, one far" else np.where(o == 2 ** 40, -2 ** 40, np.sort(o))


KINDS = ["even", "idle blocks", "falling", "any, one far", "rising, one far below"]


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("groups", [64, 65, 128, 256, 257])
def test_products(g, groups, kernel):  # noqa: F811
    for i, kind in enumerate(KINDS):
        print(f"[groups] {groups} {kind} {kernel}", flush=True)
        run_grouped(g, [0] * groups, 72, 64, trans_b=i % 2 == 0, t="bf16", kernel=kernel, offsets=offsets(kind, groups),
                    M=M, bias=True, seed=i)


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("groups", [64, 65, 128, 256, 257])
def test_gradients(g, groups, kernel):  # noqa: F811
    for i, kind in enumerate(KINDS):
        print(f"[groups] gradient {groups} {kind} {kernel}", flush=True)
        run_wgrad(g, [0] * groups, 40, 24, trans_b=i % 2 == 0, t="f16", ct="f32", kernel=kernel,
                  offsets=offsets(kind, groups), M=M, seed=i)


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("groups", [65, 128, 257])
def test_integer_products(g, groups, kernel):  # noqa: F811
    sizes = np.diff(offsets("even", groups)).tolist()
    for sizes in (sizes, [0] * (groups - 1) + [M], [M] + [0] * (groups - 1)):
        run_i8(g, sizes, 48, 64, trans_b=True, ct="bf16", kernel=kernel, bias=True, seed=groups)
