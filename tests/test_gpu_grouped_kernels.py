"""Every kernel of the grouped and 8-bit integer products by name, with the inputs, references and
tolerances of test_gpu_grouped.py: the tiled kernels where their alignment holds, the streaming
kernel at any, and the sizes at which each one's tiles, K loops and column blocks end."""
import numpy as np
import pytest

import test_gpu_grouped as base
from test_gpu_grouped import (DIMS, MANY, SIZES, check, dev, g, host, offsets_of, run_grouped,  # noqa: F401
                              run_i8, run_quantize, run_wgrad)

pytestmark = pytest.mark.gpu

TILES = [2, 3, 4]
STREAM = 5
WIDE = DIMS + [(520, 264), (64, 2048), (72, 560), (24, 40)]


def up(x, m):
    return -(-x // m) * m


@pytest.mark.parametrize("kernel", TILES + [STREAM])
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_grouped(g, t, trans_b, kernel):  # noqa: F811
    for i, sizes in enumerate(SIZES + [[16, 17, 15], [32, 33], [1000]]):
        for j, (N, K) in enumerate(WIDE):
            if kernel != STREAM:
                N, K = up(N, 8), up(K, 8)
            elif not trans_b:
                N = max(N, 4)
            print(f"[grouped] {t} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_grouped(g, sizes, N, K, trans_b=trans_b, t=t, kernel=kernel, seed=10 * i + j,
                        bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                        alpha=0.75 if j % 2 else 1.0, beta=-0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", TILES + [STREAM])
@pytest.mark.parametrize("trans_b", [False, True])
def test_grouped_strides_and_offsets(g, trans_b, kernel):  # noqa: F811
    for poison in (np.nan, np.inf):
        run_grouped(g, [40, 0, 90], 72, 104, trans_b=trans_b, t="bf16", kernel=kernel, lda=128,
                    ldb=120, ldc=80, stride=120 * 112, offsets=[7, 47, 47, 137], M=150,
                    poison=poison, bias=True, seed=3)
    run_grouped(g, [40, 9, 90], 72, 104, trans_b=trans_b, t="f16", kernel=kernel, stride=0, seed=4)
    for offsets in ([0, 50, 20, 100], [-5, 30, 300, 80], [2 ** 40, 0, 5, 9], [-2 ** 62, 2 ** 62, 3, 1]):
        run_grouped(g, [0, 0, 0], 64, 64, trans_b=trans_b, t="bf16", kernel=kernel, offsets=offsets,
                    M=100, seed=5)
    # more groups than a wave has lanes, the rows at the end, and one group of each kind
    run_grouped(g, [0] * 130 + [70, 0, 5], 64, 64, trans_b=trans_b, t="bf16", kernel=kernel, seed=6)
    run_grouped(g, [2] * 63 + [0, 300] + [1] * 80, 64, 64, trans_b=trans_b, t="bf16", kernel=kernel, seed=7)


@pytest.mark.parametrize("kernel", TILES)
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_wgrad(g, t, ct, trans_b, kernel):  # noqa: F811
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(WIDE):
            N, K = up(N, 8), up(K, 8)
            print(f"[wgrad] {t} {ct} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            if sizes is MANY and N * K > 70000:
                continue
            run_wgrad(g, sizes, N, K, trans_b=trans_b, t=t, ct=ct, kernel=kernel, seed=10 * i + j,
                      dbias=(i + j) % 3 != 0, alpha=0.5 if j % 2 else 1.0,
                      beta=1.0 if (i + j) % 2 else 0.0)
    for poison in (np.nan, np.inf):
        run_wgrad(g, [40, 0, 90], 72, 104, trans_b=trans_b, t=t, ct=ct, kernel=kernel, lda=128,
                  ldd=80, ldc=112, stride=112 * 112, offsets=[7, 47, 47, 137], M=150, poison=poison)


@pytest.mark.parametrize("kernel", TILES + [STREAM])
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_i8(g, ct, trans_b, kernel):  # noqa: F811
    for i, sizes in enumerate(SIZES + [[16, 17, 15], [32, 33], [1000], [37]]):
        for j, (N, K) in enumerate(WIDE):
            if kernel != STREAM:
                N, K = up(N, 16), up(K, 16)
            elif not trans_b:
                N = max(N, 4)
            print(f"[i8] {ct} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_i8(g, sizes, N, K, trans_b=trans_b, ct=ct, grouped=len(sizes) > 1 or j % 2 == 0,
                   kernel=kernel, seed=10 * i + j, bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                   alpha=-0.75 if j % 2 else 1.0, beta=0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", TILES + [STREAM])
@pytest.mark.parametrize("trans_b", [False, True])
def test_i8_exact_sums(g, trans_b, kernel):  # noqa: F811
    """The largest sums 31 bits hold, and sums past 24 bits: nothing is lost."""
    import torch
    for M, N, K, lda in ((2, 16, 131071, 131072), (70, 48, 8208, 8208)):
        A = torch.randint(-128, 128, (M, lda), device="cuda").to(torch.int8)
        B = torch.randint(-128, 128, (N, K), device="cuda").to(torch.int8)
        A[0], B[:8] = -128, -128
        Bs = torch.zeros(N, lda, device="cuda", dtype=torch.int8)
        Bs[:, :K] = B
        Bs = Bs if trans_b else B.t().contiguous()
        C, one = torch.zeros(M, N, device="cuda"), torch.ones(M + N, device="cuda")
        g.run_i8(A, one, Bs, one, C, M=M, N=N, K=K, lda=lda, ldb=lda if trans_b else N,
                 trans_b=trans_b, c_type="f32", kernel=kernel)
        assert torch.equal(C.cpu(), (A[:, :K].cpu().double() @ B.cpu().double().t()).float())


def test_misaligned_pointers_and_odd_rows(g):  # noqa: F811
    """8-bit and 16-bit operands from any byte or element on, with odd leading dimensions, whatever
    kernel takes them."""
    import torch
    rng = np.random.default_rng(21)
    for M, N, K in ((5, 37, 101), (70, 66, 129), (300, 131, 75)):
        for kernel in (0, 1, STREAM):
            A = dev(rng.integers(-128, 128, M * (K + 2) + 3).astype(np.int8))
            B = dev(rng.integers(-128, 128, K * (N + 1) + 5).astype(np.int8))
            sa, sb = torch.rand(M + 1, device="cuda")[1:], torch.rand(N + 1, device="cuda")[1:]
            C = torch.zeros(M * (N + 1) + 1, device="cuda", dtype=torch.float16)
            g.run_i8(A[3:], sa, B[5:], sb, C[1:], M=M, N=N, K=K, lda=K + 2, ldb=N + 1, ldc=N + 1,
                     c_type="f16", alpha=2.0 ** -12, kernel=kernel)
            a = A[3:].cpu().numpy().reshape(M, K + 2)[:, :K].astype(np.int64)
            b = B[5:].cpu().numpy().reshape(K, N + 1)[:, :N].astype(np.int64)
            ref = 2.0 ** -12 * (a @ b) * host(sa)[:, None] * host(sb)
            check(host(C[1:]).reshape(M, N + 1)[:, :N], ref, np.abs(ref), 2.0 ** -11 + 8 * 2.0 ** -24, "f16",
                  (M, N, K, kernel))
            assert not C[0] and not C[1:].view(M, N + 1)[:, N:].any()


def test_kernels_that_do_not_fit(g):  # noqa: F811
    """A kernel asked for by name refuses what it cannot do."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    A = torch.zeros(64 * 64, device="cuda", dtype=torch.bfloat16)
    C = torch.ones(64 * 64, device="cuda", dtype=torch.bfloat16)
    B = torch.zeros(64 * 64, device="cuda", dtype=torch.bfloat16)
    off = dev(np.array([0, 8], dtype=np.int64))

    def refused(status, **kw):
        a = dict(groups=1, M=8, N=16, K=16)
        a.update(kw)
        with pytest.raises(tmm.GemmError) as e:
            g.run_grouped(A[a.pop("skew", 0):], B, C, off, **a)
        assert e.value.status == status

    for k in TILES:
        refused(tmm.GEMM_ERR_UNSUPPORTED, kernel=k, skew=1)
        refused(tmm.GEMM_ERR_UNSUPPORTED, kernel=k, K=12, lda=12)
        refused(tmm.GEMM_ERR_UNSUPPORTED, kernel=k, N=12, ldb=12)
    refused(tmm.GEMM_ERR_UNSUPPORTED, kernel=STREAM, N=3)
    refused(tmm.GEMM_ERR_INVALID_VALUE, kernel=6)
    refused(tmm.GEMM_ERR_INVALID_VALUE, kernel=-1)
    with pytest.raises(tmm.GemmError):
        g.run_grouped_wgrad(A, B, C, off, groups=1, M=8, N=16, K=16, kernel=STREAM)
    torch.cuda.synchronize()
    assert (C == 1).all()


@pytest.mark.parametrize("kernel", [0, 1] + TILES + [STREAM])
def test_nothing_to_sum(g, kernel):  # noqa: F811
    """K = 0: the epilogue of zero sums; a gradient without columns still has its bias gradient."""
    for trans_b in (False, True):
        run_grouped(g, [5, 0, 70], 48, 0, trans_b=trans_b, t="bf16", kernel=kernel, lda=8, ldb=48,
                    stride=0, bias=True, do_gelu=True, beta=0.5)
        run_i8(g, [5, 0, 70], 48, 0, trans_b=trans_b, ct="f16", kernel=kernel, lda=16, ldb=48, bias=True)
    if kernel != STREAM:
        import torch
        D = torch.randn(9, 24, device="cuda").to(torch.bfloat16)
        db = torch.full((2, 24), float("nan"), device="cuda")
        g.run_grouped_wgrad(None, D, None, dev(np.array([0, 4, 9], dtype=np.int64)), groups=2, M=9, N=24,
                            K=0, lda=8, ldc=24, dbias=db, kernel=kernel)
        want = np.stack([host(D)[:4].sum(0), host(D)[4:].sum(0)])
        size = np.stack([np.abs(host(D))[:4].sum(0), np.abs(host(D))[4:].sum(0)])
        check(host(db), want, size, 9 * 2.0 ** -24, "f32", kernel)


@pytest.mark.parametrize("kernel", TILES + [STREAM])
def test_far_addresses(g, kernel):  # noqa: F811
    base.test_grouped_far_addresses(g, kernel)


@pytest.mark.parametrize("kernel", TILES + [STREAM])
def test_infinities_stay_in_their_rows(g, kernel):  # noqa: F811
    base.test_grouped_infinities_stay_in_their_rows(g, kernel)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_quantize_lengths(g, t):  # noqa: F811
    """Rows that end at every place of the threads' chunks: one wave, four waves, past the registers."""
    rng = np.random.default_rng(22)
    for K in (4, 15, 16, 255, 256, 257, 1023, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 8191, 8192, 8193,
              16383, 16384, 16390, 33000):
        for M in (1, 5):
            print(f"[quantize] {t} {M} {K}", flush=True)
            x = rng.standard_normal((M, K))
            x[:, K - 1] = 5.0  # the last element decides the scale
            run_quantize(g, x, t, ldx=K + K % 3)
