"""Paths of the grouped MXFP4 tiles that only some calls take: widths that are no multiple of 4 in rows of C that
are (a tile's last columns one by one), and the mixed kernel's 256 x 256 tiles, which it keeps whole from more
than half a round of the compute units on.  Tolerances are test_gpu_experts.py's."""
import pytest

from test_gpu_experts import TILES, g, run_mx  # noqa: F401
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
