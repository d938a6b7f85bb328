"""Grouped products and gradients whose workgroups have 2^32 work items or more between them, more
than one launch takes.  Small whole numbers, so that every result is exact."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tiled_matrix_multiply_amd as tmm
    h = tmm.Gemm(0)
    yield h
    h.close()
    torch.cuda.empty_cache()


def whole(gen, *shape):
    import torch
    return torch.randint(-1, 2, shape, device="cuda", generator=gen, dtype=torch.int8).to(torch.bfloat16)


# 1024 groups of one row, one matrix for all of them (stride 0): a workgroup for every 32 columns
# (streamed) or 64 (tiles) of each row
@pytest.mark.parametrize("kernel,N,threads,columns", [(0, 2 ** 18 + 64, 512, 32), (5, 2 ** 18 + 64, 512, 32),
                                                      (1, 2 ** 20 + 64, 256, 64), (2, 2 ** 19 + 64, 512, 64)])
def test_products(g, kernel, N, threads, columns):
    import torch
    G = M = 1024
    K = 8
    assert G * (N // columns) * threads >= 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(kernel)
    A, B = whole(gen, M, K), whole(gen, N, K)
    C = torch.full((M, N), 77.0, device="cuda", dtype=torch.bfloat16)
    off = torch.arange(G + 1, device="cuda")
    print(f"[many workgroups] kernel {kernel} N {N}", flush=True)
    g.run_grouped(A, B, C, off, groups=G, M=M, N=N, K=K, trans_b=True, stride_b=0, kernel=kernel)
    a, b = A.float(), B.float()
    for n in range(0, N, 2 ** 17):
        cols = slice(n, min(N, n + 2 ** 17))
        assert torch.equal(C[:, cols].float(), a @ b[cols].t()), n


def test_gradient(g):
    """64 groups of one row and one channel of input: 2^24 workgroups, half of them for the bias."""
    import torch
    G = M = 64
    N, K = 2 ** 23 + 64, 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    A, D = whole(gen, M, K), whole(gen, M, N)
    C = torch.full((G, K, N), 77.0, device="cuda", dtype=torch.bfloat16)
    db = torch.full((G, N), 77.0, device="cuda")
    off = torch.arange(G + 1, device="cuda")
    print("[many workgroups] gradient", flush=True)
    g.run_grouped_wgrad(A, D, C, off, groups=G, M=M, N=N, K=K, dbias=db)
    for q in range(G):
        assert torch.equal(C[q, 0].float(), A[q].float() * D[q].float()), q
        assert torch.equal(db[q], D[q].float()), q
