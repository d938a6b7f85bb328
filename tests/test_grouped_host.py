"""The entry points of include/gemm_grouped.h without a GPU: every declared symbol is exported and
bound, and argument checks answer as the header states."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
tmm = pytest.importorskip("tiled_matrix_multiply_amd")

F32, F16, BF16, E4M3 = tmm.GEMM_F32, tmm.GEMM_F16, tmm.GEMM_BF16, tmm.GEMM_E4M3
OK, V, U, AL, NH = (tmm.GEMM_OK, tmm.GEMM_ERR_INVALID_VALUE, tmm.GEMM_ERR_UNSUPPORTED,
                    tmm.GEMM_ERR_ALIAS, tmm.GEMM_ERR_INVALID_HANDLE)
BIAS, GELU = tmm.GEMM_EPI_BIAS, tmm.GEMM_EPI_GELU
# Fake, well-separated device addresses: the checks never dereference them.
PO, PA, PB, PC, PSA, PSB, PBIAS = (0x10000000 * i for i in range(1, 8))


def test_symbols_are_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "gemm_grouped.h")).read()
    syms = sorted(set(re.findall(r"GEMM_API\s+[\w\s\*]*?\b(gemm_\w+)\s*\(", text)))
    assert sorted(tmm.GROUPED_EXPORTS) == syms
    for s in syms:
        assert hasattr(tmm.library(), s) and hasattr(tmm, s)


def test_kernel_names_match_the_header():
    text = open(os.path.join(ROOT, "include", "gemm_grouped.h")).read()
    enum = dict(re.findall(r"\b(GEMM_GROUPED_\w+) = (\d+)", text))
    assert {int(v) for v in enum.values()} == set(tmm.GROUPED_KERNEL_NAME)
    for name, v in enum.items():
        assert getattr(tmm, name) == int(v)


def chk(G=3, off=PO, M=40, N=48, K=64, tb=0, A=PA, lda=None, sa=None, B=PB, ldb=None, stride=None,
        sb=None, C=PC, ldc=None, i8=0, t=BF16, ct=None, epi=0, bias=None):
    lda = K if lda is None else lda
    ldb = (K if tb else N) if ldb is None else ldb
    stride = (N if tb else K) * ldb if stride is None else stride
    if i8:
        sa = PSA if sa is None else sa or None
        sb = PSB if sb is None else sb or None
    return tmm.gemm_check_args_grouped(G, off, M, N, K, tb, A, lda, sa, B, ldb, stride, sb, C,
                                       N if ldc is None else ldc, i8, t, t if ct is None else ct,
                                       epi, bias)


@pytest.mark.parametrize("i8", [0, 1])
def test_products(i8):
    for tb in (0, 1):
        for t in (F16, BF16):
            assert chk(i8=i8, tb=tb, t=t) == OK
            assert chk(i8=i8, tb=tb, t=t, epi=BIAS | GELU, bias=PBIAS) == OK
    assert chk(i8=i8, M=-1) == V and chk(i8=i8, N=-1, ldc=1) == V and chk(i8=i8, K=-1) == V
    assert chk(i8=i8, G=-1) == V and chk(i8=i8, tb=2) == V and chk(i8=i8, epi=4) == V
    assert chk(i8=i8, off=None) == V
    assert chk(i8=i8, off=PO + 4) == V                       # not a place for 64-bit numbers
    assert chk(i8=i8, A=None) == V and chk(i8=i8, B=None) == V and chk(i8=i8, C=None) == V
    assert chk(i8=i8, lda=63) == V and chk(i8=i8, ldb=47) == V and chk(i8=i8, tb=1, ldb=63) == V
    assert chk(i8=i8, ldc=47) == V and chk(i8=i8, stride=-1) == V
    assert chk(i8=i8, stride=0) == OK                        # one matrix for every group
    assert chk(i8=i8, epi=BIAS) == V
    assert chk(i8=i8, G=65535, stride=0) == OK and chk(i8=i8, G=65536, stride=0) == U
    assert chk(i8=i8, M=2 ** 31) == U and chk(i8=i8, N=2 ** 31) == U
    # nothing to compute
    assert chk(i8=i8, M=0, A=None, C=None, off=None) == OK
    assert chk(i8=i8, N=0, C=None, B=None) == OK and chk(i8=i8, G=0, off=None) == OK
    assert chk(i8=i8, K=0, A=None, B=None, lda=0, ldb=48) == OK
    # C (40 x 48, 2 bytes each) against everything that is read
    size = 40 * 48 * 2
    es = 1 if i8 else 2
    assert chk(i8=i8, C=PA) == AL and chk(i8=i8, C=PB) == AL and chk(i8=i8, C=PO) == AL
    assert chk(i8=i8, C=PA - size) == OK and chk(i8=i8, C=PA - size + 1) == AL
    assert chk(i8=i8, C=PB + 3 * 48 * 64 * es - 1) == AL      # the last group's matrix
    assert chk(i8=i8, C=PB + 3 * 48 * 64 * es) == OK
    assert chk(i8=i8, C=PO + 31) == AL and chk(i8=i8, C=PO + 32) == OK
    assert chk(i8=i8, epi=BIAS, bias=PC + size - 4) == AL
    assert chk(i8=i8, epi=BIAS, bias=PC - 3 * 48 * 4 + 4) == AL
    assert chk(i8=i8, epi=BIAS, bias=PC - 3 * 48 * 4) == OK


def test_types():
    assert chk(t=F32) == U and chk(t=E4M3) == U and chk(t=BF16, ct=F16) == U and chk(t=F16, ct=F32) == U
    for ct in (F16, BF16, F32):
        assert chk(i8=1, t=99, ct=ct) == OK
    assert chk(i8=1, ct=E4M3) == U


def test_integer_products():
    assert chk(i8=1, sa=0) == V and chk(i8=1, sb=0) == V
    assert chk(i8=1, K=131071) == OK and chk(i8=1, K=131072) == U
    assert chk(i8=1, C=PSA + 159) == AL and chk(i8=1, C=PSA + 160) == OK
    assert chk(i8=1, C=PSB + 3 * 48 * 4 - 1) == AL and chk(i8=1, C=PSB + 3 * 48 * 4) == OK
    assert chk(i8=1, G=1, off=None) == OK                    # gemm_run_i8


def chk_w(G=3, off=PO, M=40, N=48, K=64, tb=0, A=PA, lda=None, D=PB, ldd=None, C=PC, ldc=None,
          stride=None, t=BF16, ct=None, db=None):
    ldc = (K if tb else N) if ldc is None else ldc
    stride = (N if tb else K) * ldc if stride is None else stride
    return tmm.gemm_check_args_grouped_wgrad(G, off, M, N, K, tb, A, K if lda is None else lda, D,
                                             N if ldd is None else ldd, C, ldc, stride, t,
                                             t if ct is None else ct, db)


def test_weight_gradient():
    for tb in (0, 1):
        for t in (F16, BF16):
            assert chk_w(tb=tb, t=t) == OK and chk_w(tb=tb, t=t, ct=F32, db=PBIAS) == OK
    assert chk_w(t=F32) == U and chk_w(t=F16, ct=BF16) == U and chk_w(G=65536) == U
    assert chk_w(M=-1) == V and chk_w(G=-1) == V and chk_w(tb=3) == V
    assert chk_w(off=None) == V and chk_w(A=None) == V and chk_w(D=None) == V and chk_w(C=None) == V
    assert chk_w(lda=63) == V and chk_w(ldd=47) == V and chk_w(ldc=47) == V
    assert chk_w(tb=1, ldc=63) == V
    assert chk_w(stride=64 * 48 - 1) == V and chk_w(G=1, stride=0) == OK
    assert chk_w(M=0, A=None, D=None) == OK and chk_w(N=0, C=None) == OK
    assert chk_w(K=0, A=None, C=None) == OK                          # nothing to compute
    assert chk_w(K=0, A=None, C=None, D=None, db=PBIAS) == V         # dbias reads D
    assert chk_w(K=0, A=None, C=None, db=PBIAS) == OK
    size = 3 * 64 * 48 * 2
    assert chk_w(C=PA) == AL and chk_w(C=PB + 40 * 48 * 2 - 1) == AL and chk_w(C=PB + 40 * 48 * 2) == OK
    assert chk_w(C=PO) == AL
    assert chk_w(db=PC + size - 1) == AL and chk_w(db=PC + size) == OK
    assert chk_w(db=PA) == AL and chk_w(db=PB) == AL and chk_w(db=PO) == AL


def chk_z(M=40, K=64, X=PA, ldx=None, t=BF16, Q=PB, ldq=None, s=PC):
    return tmm.gemm_check_args_quantize_rows(M, K, X, K if ldx is None else ldx, t, Q,
                                             K if ldq is None else ldq, s)


def test_quantize_rows():
    for t in (F32, F16, BF16):
        assert chk_z(t=t) == OK
    assert chk_z(t=E4M3) == U and chk_z(M=2 ** 31) == U
    assert chk_z(M=-1) == V and chk_z(K=-1) == V
    assert chk_z(X=None) == V and chk_z(Q=None) == V and chk_z(s=None) == V
    assert chk_z(ldx=63) == V and chk_z(ldq=63) == V
    assert chk_z(M=0, X=None, Q=None, s=None) == OK and chk_z(K=0, X=None, Q=None) == OK
    assert chk_z(Q=PA + 40 * 64 * 2 - 1) == AL and chk_z(Q=PA + 40 * 64 * 2) == OK
    assert chk_z(s=PA) == AL and chk_z(s=PB + 40 * 64 - 4) == AL and chk_z(Q=PC + 8) == AL


def test_null_handle():
    assert tmm.gemm_run_grouped(None, 0, None, 1, PO, 4, 4, 4, 0, 1.0, PA, 4, PB, 4, 16, 0.0, PC, 4,
                                BF16, 0, None) == NH
    assert tmm.gemm_run_grouped_wgrad(None, 0, None, 1, PO, 4, 4, 4, 0, 1.0, PA, 4, PB, 4, 0.0, PC,
                                      4, 16, BF16, BF16, None) == NH
    assert tmm.gemm_run_i8(None, 0, None, 4, 4, 4, 0, 1.0, PA, 4, PSA, PB, 4, PSB, 0.0, PC, 4, BF16,
                           0, None) == NH
    assert tmm.gemm_run_grouped_i8(None, 0, None, 1, PO, 4, 4, 4, 0, 1.0, PA, 4, PSA, PB, 4, 16, PSB,
                                   0.0, PC, 4, BF16, 0, None) == NH
    assert tmm.gemm_run_grouped_i8(None, 0, None, 1, None, 4, 4, 4, 0, 1.0, PA, 4, PSA, PB, 4, 16,
                                   PSB, 0.0, PC, 4, BF16, 0, None) == NH
    assert tmm.gemm_quantize_rows(None, None, 4, 4, PA, 4, BF16, PB, 4, PC) == NH
