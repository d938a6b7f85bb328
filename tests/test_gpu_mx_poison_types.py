"""The LDS race check of test_gpu_experts_poison.py for the grouped MXFP4 tiles with fp16 and fp32 results, whose
tiles have registers of their own, and at the sizes where the mixed kernel keeps 256 x 256 tiles whole, splits
some, and gives a workgroup a second tile."""
import numpy as np
import pytest

from test_gpu_experts_poison import handles  # noqa: F401
from test_gpu_grouped_paths import MIXED, compute_units, dtype, mixed

pytestmark = pytest.mark.gpu


def both(handles, ct, sizes, N, K, kernel, do_gelu):  # noqa: F811
    """The bits of the library and of the check's build for one call."""
    import torch
    tmm, using, dbg, g, gd = handles
    rng = np.random.default_rng([K, N])
    G, M, lds = len(sizes), sum(sizes), (K // 32 + 15) // 16 * 16
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), device="cuda")

    def some(lo, hi, *shape):
        return torch.from_numpy(rng.integers(lo, hi, shape).astype(np.uint8)).cuda()

    A, B, sa, sb = some(0, 256, M, K // 2), some(0, 256, G, N, K // 2), some(123, 132, M, lds), some(123, 132, G, N, lds)
    bias = torch.randn(G, N, device="cuda")

    def call(h):
        C = torch.full((M, N), 7.0, device="cuda", dtype=dtype(ct))
        h.run_grouped_mx(A, sa, B, sb, C, off, groups=G, M=M, N=N, K=K, c_type=ct, kernel=kernel, bias=bias, alpha=2.0 ** -6,
                         beta=0.5, epilogue=tmm.GEMM_EPI_BIAS | (tmm.GEMM_EPI_GELU if do_gelu else 0), ldsa=lds, ldsb=lds)
        torch.cuda.synchronize()
        return C

    print(f"[mx poison] {ct} {kernel} {sizes[:4]} {N} {K}", flush=True)
    want = call(g)
    with using(dbg):
        got = call(gd)
    assert torch.equal(got, want) and bool(want.isfinite().all()), (ct, kernel, sizes, N, K)


@pytest.mark.parametrize("kernel,K", [(2, 32), (2, 1056), (2, 4128), (2, 5152), (3, 96), (3, 544), (3, 2080), (4, 64), (4, 544),
                                      (4, 2080)])
@pytest.mark.parametrize("ct", ["f16", "f32"])
def test_poisoned_stages_change_nothing(handles, ct, kernel, K):  # noqa: F811
    for sizes in ([300, 0, 70, 513], [1100]):
        for N in (64, 520):
            both(handles, ct, sizes, N, K, kernel, N == 64)


@pytest.mark.parametrize("path", sorted(MIXED))
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_poisoned_stages_of_the_mixed_kernel(handles, ct, path):  # noqa: F811
    sizes, N = MIXED[path]
    if compute_units() == 256:
        assert mixed(sizes, N, 256)[0] > 128
    for K in (256, 544, 2080):
        both(handles, ct, sizes, N, K, 4, K == 544)
