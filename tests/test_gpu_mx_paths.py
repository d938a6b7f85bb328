"""Paths of the grouped MXFP4 tiles that only some calls take: widths that are no multiple of 4 in rows of C that
are (a tile's last columns one by one), and the mixed kernel's 256 x 256 tiles, which it keeps whole from more
than half a round of the compute units on.  Tolerances are test_gpu_experts.py's."""
import numpy as np
import pytest

from test_gpu_experts import RNG, STREAM, TILES, U32, check, dev, g, host, random_mx, run_mx, unpack, values  # noqa: F401
from test_gpu_grouped_paths import MIXED, compute_units, mixed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [0] + TILES)
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_mx_widths(g, ct, kernel):  # noqa: F811
    for i, sizes in enumerate([[5, 0, 7], [64, 65, 1, 0, 127], [300, 2, 513]]):
        for j, N in enumerate((1, 2, 3, 5, 33, 63, 65, 127, 130, 259)):
            print(f"[mx] width {ct} {kernel} {sizes} {N}", flush=True)
            run_mx(g, sizes, N, 96 if j % 2 else 544, ct=ct, kernel=kernel, ldc=(N + 3) // 4 * 4 + 4 * (i % 2), seed=i + j,
                   bias=(i + j) % 2 == 0, do_gelu=j % 3 == 0, alpha=0.75, beta=-0.5 if j % 4 < 2 else 0.0)


@pytest.mark.parametrize("N", [4101, 2050])
def test_mx_wide_and_odd(g, N):  # noqa: F811
    """As AUTO takes them: prompts and few rows of a layer whose width is odd, in padded rows."""
    for sizes in ([37], [700], [256, 130, 3, 311]):
        for ct in ("bf16", "f16"):
            print(f"[mx] odd {sizes} {N} {ct}", flush=True)
            run_mx(g, sizes, N, 544, ct=ct, ldc=N + 4 - N % 4, bias=True, do_gelu=True, seed=N, no_offsets=len(sizes) == 1)


@pytest.mark.parametrize("path", sorted(MIXED))
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_mx_mixed(g, ct, path):  # noqa: F811
    sizes, N = MIXED[path]
    kept, split, pieces = mixed(sizes, N, compute_units())
    if compute_units() == 256:
        assert kept > 128 and (split > 0) == (path != "kept")
        assert (pieces > 256) == (path == "more pieces than workgroups")
    # 2 K tiles, the last one cut, and 5
    for K, do_gelu, beta, kernel in ((288, False, -0.5, 4), (1056, True, 0.0, 0 if path != "kept" else 4)):
        print(f"[mx] mixed {path} {ct} {K}", flush=True)
        run_mx(g, sizes, N, K, ct=ct, kernel=kernel, bias=True, do_gelu=do_gelu, beta=beta, seed=K, ldc=N + 8)


@pytest.mark.parametrize("kernel", [STREAM] + TILES)
def test_mx_scales_at_the_ends(g, kernel):  # noqa: F811
    """The smallest scales of one operand with the largest of the other, and blocks of zeros, whose scale byte is
    0: products are exact, sums within K 2^-23 of sum |a b|."""
    import torch
    rng = RNG(kernel)
    M, N, K = 70, 40, 544
    for low_a in (True, False):
        qa, _, _ = random_mx(rng, M, K, K, 32)
        qb, _, _ = random_mx(rng, N, K, K, 32)
        low, high = (rng.integers(0, 4, (n, 32)).astype(np.uint8) for n in ((M, N) if low_a else (N, M)))
        high = 254 - high
        sa, sb = (low, high) if low_a else (high, low)
        qa[:, 32:64], sa[:, 2:4] = 0, 0                                  # two blocks of zeros
        a, b = values(unpack(qa), sa[:, :K // 32]), values(unpack(qb), sb[:, :K // 32])
        C = torch.full((M, N), 7.0, device="cuda:0")
        g.run_grouped_mx(dev(qa), dev(sa), dev(qb), dev(sb), C, None, groups=1, M=M, N=N, K=K, c_type="f32", ldsa=32,
                         ldsb=32, kernel=kernel)
        torch.cuda.synchronize()
        check(host(C), a @ b.T, (K * 2.0 ** -23 + 4 * U32) * (np.abs(a) @ np.abs(b).T), "f32", (kernel, low_a))
