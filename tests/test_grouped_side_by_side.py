"""Weight gradients whose matrices lie side by side in the rows of one (K, or with transB N, x groups x
row elements), the layout of a B whose groups do: the argument checks, and the values on the GPU."""
import numpy as np
import pytest

tmm = pytest.importorskip("tiled_matrix_multiply_amd")

OK, V, AL = tmm.GEMM_OK, tmm.GEMM_ERR_INVALID_VALUE, tmm.GEMM_ERR_ALIAS
PO, PA, PB, PC = (0x10000000 * i for i in range(1, 5))


def test_checks():
    def chk(G, ldc, stride, tb=0, N=48, K=64, C=PC):
        return tmm.gemm_check_args_grouped_wgrad(G, PO, 40, N, K, tb, PA, K, PB, N, C, ldc, stride,
                                                 tmm.GEMM_BF16, tmm.GEMM_BF16, None)

    for tb, row in ((0, 48), (1, 64)):
        assert chk(3, 3 * row, row, tb) == OK and chk(3, 3 * row + 1, row, tb) == OK
        assert chk(3, 3 * row - 1, row, tb) == V            # the last matrix leaves the rows
        assert chk(3, 3 * row, row - 1, tb) == V            # neighbours share elements
        assert chk(3, 4 * row, row + row // 2, tb) == OK and chk(3, 4 * row - 1, row + row // 2, tb) == V
        assert chk(65535, 65535 * row, row, tb) == OK and chk(1, row, 0, tb) == OK
        assert chk(3, 3 * row, 0, tb) == V and chk(3, 3 * row, -row, tb) == V
    # the whole extent counts against the operands: 64 rows of 144 elements of 2 bytes
    assert chk(3, 144, 48, C=PB - 64 * 144 * 2 + 1) == AL and chk(3, 144, 48, C=PB - 64 * 144 * 2) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f32")])
def test_values(t, ct, trans_b, kernel):
    """The bits are those of the gradient with the matrices one after another."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    types = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    sizes = [40, 0, 90, 300]
    G, M = len(sizes), sum(sizes)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).cuda()
    for N, K, gap in ((72, 104, 8), (264, 520, 0), (64, 64, 0)):
        gen = torch.Generator(device="cuda").manual_seed(N)
        A = torch.randn(M, K, device="cuda", generator=gen).to(types[t])
        D = torch.randn(M, N, device="cuda", generator=gen).to(types[t])
        rows, cols = (N, K) if trans_b else (K, N)
        start = torch.randn(G, rows, cols, device="cuda", generator=gen).to(types[ct])
        one, wide = start.clone(), torch.full((rows, G, cols + gap), 3.0, device="cuda", dtype=types[ct])
        wide[:, :, :cols] = start.transpose(0, 1)
        kw = dict(groups=G, M=M, N=N, K=K, trans_b=trans_b, a_type=t, c_type=ct, alpha=0.5, beta=-1.0, kernel=kernel)
        with tmm.Gemm(0) as g:
            g.run_grouped_wgrad(A, D, one, off, **kw)
            g.run_grouped_wgrad(A, D, wide, off, ldc=G * (cols + gap), stride_c=cols + gap, **kw)
            torch.cuda.synchronize()
        assert torch.equal(wide[:, :, :cols].transpose(0, 1), one), (N, K)
        assert (wide[:, :, cols:] == 3.0).all()
        assert not torch.equal(one[0], start[0]) and torch.equal(one[1], -start[1])
