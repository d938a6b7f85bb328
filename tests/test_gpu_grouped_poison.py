"""LDS race check of the grouped and 8-bit integer products (the method of test_gpu_lds_poison.py):
the build whose kernels overwrite every LDS stage with all-ones words before refilling it has to give
the library's bits on every tiled kernel, with short, ragged and empty groups and K loops of one, two
and many tiles."""
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
    for name in tmm.EXPORTS + tmm.GROUPED_EXPORTS:
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


SIZES = [[300, 0, 70, 513], [256, 128, 1], [1100]]


@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
@pytest.mark.parametrize("trans_b", [False, True])
def test_poisoned_stages_change_nothing(handles, kernel, trans_b):
    import torch
    tmm, using, dbg, g, gd = handles
    rng = np.random.default_rng(31)
    for sizes in SIZES:
        for N, K in ((272, 64), (520, 208), (128, 1040)):
            G, M = len(sizes), sum(sizes)
            off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), device="cuda")
            A = torch.randn(M, K, device="cuda").to(torch.bfloat16)
            D = torch.randn(M, N, device="cuda").to(torch.bfloat16)
            B = torch.randn(G, N * K, device="cuda").to(torch.bfloat16)
            A8 = torch.from_numpy(rng.integers(-128, 128, (M, K)).astype(np.int8)).cuda()
            B8 = torch.from_numpy(rng.integers(-128, 128, (G, N * K)).astype(np.int8)).cuda()
            sa, sb = torch.rand(M, device="cuda"), torch.rand(G, N, device="cuda")
            print(f"[poison] {kernel} {trans_b} {sizes} {N} {K}", flush=True)

            def call(h):
                C, C8 = (torch.full((M, N), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
                W = torch.full((G, N * K), 7.0, device="cuda")
                db = torch.zeros(G, N, device="cuda")
                kw = dict(groups=G, M=M, N=N, K=K, trans_b=trans_b, kernel=kernel)
                h.run_grouped(A, B, C, off, **kw)
                if (N if not trans_b else K) % 16 == 0 or kernel == 1:
                    h.run_grouped_i8(A8, sa, B8, sb, C8, off, **kw)
                h.run_grouped_wgrad(A, D, W, off, c_type="f32", dbias=db, **kw)
                torch.cuda.synchronize()
                return C, C8, W, db

            want = call(g)
            with using(dbg):
                got = call(gd)
            for a, b in zip(want, got):
                assert torch.equal(a, b) and not torch.isnan(a).any(), (kernel, trans_b, sizes, N, K)
