"""LDS race check of the grouped MXFP4 tiles (the method of test_gpu_lds_poison.py): the build whose
kernels overwrite every LDS stage, data and block scales, with all-ones words before refilling it has to
give the library's bits on every tiled kernel, with short, ragged and empty groups and K loops of one,
two and many tiles."""
import contextlib
import ctypes
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handles():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tiled_matrix_multiply_amd as tmm
    path = os.path.join(os.path.dirname(tmm.LIB_PATH), "libgemm_lds_poison.so")
    assert os.path.exists(path), f"{path} is missing: build the library first"
    dbg = ctypes.CDLL(path)
    for name in tmm.EXPORTS + tmm.EXPERTS_EXPORTS:
        src, dst = getattr(tmm.library(), name), getattr(dbg, name)
        dst.argtypes, dst.restype = src.argtypes, src.restype

    @contextlib.contextmanager
    def using(lib):
        saved, tmm._lib = tmm._lib, lib
        try:
            yield
        finally:
            tmm._lib = saved

    g = tmm.Gemm(0)
    with using(dbg):
        gd = tmm.Gemm(0)
    yield tmm, using, dbg, g, gd
    with using(dbg):
        gd.close()
    g.close()


# (kernel, K): a K tile has 256 elements; 4128 and 5152 take the third stage of the 64 x 64 tile where there
# are few of them
@pytest.mark.parametrize("kernel,K", [(2, 32), (2, 1056), (2, 4128), (2, 5152), (3, 96), (3, 544), (3, 2080),
                                      (4, 64), (4, 544), (4, 2080)])
def test_poisoned_stages_change_nothing(handles, kernel, K):
    import torch
    tmm, using, dbg, g, gd = handles
    rng = np.random.default_rng([kernel, K])
    for sizes in ([300, 0, 70, 513], [256, 128, 1], [1100]):
        for N in (64, 272, 520):
            print(f"[mx poison] {kernel} {K} {sizes} {N}", flush=True)
            G, M, ld, lds = len(sizes), sum(sizes), K, (K // 32 + 15) // 16 * 16
            off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), device="cuda")

            def codes(*shape):
                return torch.from_numpy(rng.integers(0, 256, shape).astype(np.uint8)).cuda()

            def scales(*shape):
                return torch.from_numpy(rng.integers(123, 132, shape).astype(np.uint8)).cuda()

            A, B, sa, sb = codes(M, ld // 2), codes(G, N, ld // 2), scales(M, lds), scales(G, N, lds)
            bias = torch.randn(G, N, device="cuda")

            def call(h):
                C = torch.full((M, N), 7.0, device="cuda", dtype=torch.bfloat16)
                h.run_grouped_mx(A, sa, B, sb, C, off, groups=G, M=M, N=N, K=K, kernel=kernel, bias=bias,
                                 epilogue=tmm.GEMM_EPI_BIAS, ldsa=lds, ldsb=lds)
                torch.cuda.synchronize()
                return C

            want = call(g)
            with using(dbg):
                got = call(gd)
            assert torch.equal(got, want) and not torch.isnan(want).any(), (kernel, sizes, N, K)
