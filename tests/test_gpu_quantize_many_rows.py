"""gemm_quantize_rows with more rows than one launch's work items can count (2^32 of them): from 2^26
rows on where a wave takes a row, from 2^24 on where four do.  Codes and scales have to equal the
definition's, in 64 bits."""
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


def definition(x):
    import torch
    x = x.double()
    s = (x.abs().amax(dim=1) / 127).float()
    d = torch.where(s > 0, s, torch.ones_like(s)).double()
    return torch.round(x / d[:, None]).to(torch.int8), s


def test_rows_of_a_wave(g):
    import torch
    M, K = 2 ** 26 + 77, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(M, K, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    Q = torch.full((M, K), 99, device="cuda", dtype=torch.int8)
    s = torch.full((M,), -1.0, device="cuda")
    g.quantize_rows(X, Q, s, M=M, K=K)
    for r in range(0, M, 2 ** 24):
        rows = slice(r, min(M, r + 2 ** 24))
        q, want = definition(X[rows])
        assert torch.equal(s[rows], want) and torch.equal(Q[rows], q), r


def test_rows_of_a_workgroup(g):
    """69 GB of rows, of which those around the start, the border and the end are looked at."""
    import torch
    M, K = 2 ** 24 + 77, 1028
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("less than 100 GiB free")
    gen = torch.Generator(device="cuda").manual_seed(2)
    X = torch.empty(M, K, device="cuda")
    Q = torch.empty(M, K, device="cuda", dtype=torch.int8)
    s = torch.full((M,), -1.0, device="cuda")
    looked = [slice(0, 100), slice(2 ** 24 - 200, M)]
    for rows in looked:
        X[rows].normal_(generator=gen)
        Q[rows] = 99
    g.quantize_rows(X, Q, s, M=M, K=K, x_type="f32")
    for rows in looked:
        q, want = definition(X[rows])
        assert torch.equal(s[rows], want) and torch.equal(Q[rows], q), rows
