"""The LDS race check of test_gpu_grouped_poison.py at the sizes where the mixed kernel keeps 256 x 256
tiles whole, splits some, and gives a workgroup a second tile, and where the any-alignment tile does
not split K, in every type."""
import numpy as np
import pytest

from test_gpu_grouped_paths import MIXED, compute_units, dtype, mixed
from test_gpu_grouped_poison import handles  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", sorted(MIXED) + ["any alignment"])
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16"), ("i8", "f32")])
def test_poisoned_stages_change_nothing(handles, t, ct, nk, path):  # noqa: F811
    import torch
    tmm, using, dbg, g, gd = handles
    if path == "any alignment":
        sizes, N, depths, kernel = [700, 1, 613], 1001, (75, 1003), 1
    else:
        sizes, N = MIXED[path]
        step = 16 if t == "i8" else 8
        N, depths, kernel = -(-N // step) * step, (13 * step, 57 * step), 4
        if compute_units() == 256:
            assert mixed(sizes, N, 256)[0] > 128
    G, M = len(sizes), sum(sizes)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)).cuda()
    for K in depths:
        gen = torch.Generator(device="cuda").manual_seed(K)
        if t == "i8":
            A, B = (torch.randint(-128, 128, s, device="cuda", generator=gen, dtype=torch.int8)
                    for s in ((M, K), (G, N * K)))
        else:
            A, B = (torch.randn(*s, device="cuda", generator=gen).to(dtype(t)) for s in ((M, K), (G, N * K)))
        sa, sb = torch.rand(M, device="cuda", generator=gen), torch.rand(G, N, device="cuda", generator=gen)
        print(f"[poison] {path} {t} {ct} {nk} {K}", flush=True)

        def call(h):
            C = torch.full((M, N), 7.0, device="cuda", dtype=dtype(ct))
            kw = dict(groups=G, M=M, N=N, K=K, trans_b=nk, kernel=kernel)
            if t == "i8":
                h.run_grouped_i8(A, sa, B, sb, C, off, c_type=ct, alpha=2.0 ** -12, **kw)
            else:
                h.run_grouped(A, B, C, off, a_type=t, **kw)
            torch.cuda.synchronize()
            return C

        want = call(g)
        with using(dbg):
            got = call(gd)
        assert torch.equal(want, got) and bool(want.isfinite().all()), K


@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
def test_gradients_in_fp16(handles, kernel):  # noqa: F811
    import torch
    tmm, using, dbg, g, gd = handles
    sizes = [300, 0, 70, 513]
    G, M = len(sizes), sum(sizes)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)).cuda()
    for N, K in ((272, 64), (520, 208)):
        gen = torch.Generator(device="cuda").manual_seed(N)
        A = torch.randn(M, K, device="cuda", generator=gen).to(torch.float16)
        D = torch.randn(M, N, device="cuda", generator=gen).to(torch.float16)
        for nk in (False, True):
            for ct in ("f16", "f32"):
                def call(h):
                    W = torch.full((G, N * K), 7.0, device="cuda", dtype=dtype(ct))
                    db = torch.zeros(G, N, device="cuda")
                    h.run_grouped_wgrad(A, D, W, off, groups=G, M=M, N=N, K=K, trans_b=nk, a_type="f16", c_type=ct,
                                        dbias=db, kernel=kernel)
                    torch.cuda.synchronize()
                    return W, db

                print(f"[poison] gradient {kernel} {N} {K} {nk} {ct}", flush=True)
                want = call(g)
                with using(dbg):
                    got = call(gd)
                assert all(torch.equal(a, b) for a, b in zip(want, got)) and bool(want[0].isfinite().all())
