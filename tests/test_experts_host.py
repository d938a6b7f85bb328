"""The entry points of include/gemm_experts.h without a GPU: every declared symbol is exported and bound,
and argument checks answer as the header states."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
tmm = pytest.importorskip("tiled_matrix_multiply_amd")

F32, F16, BF16, E4M3, E2M1 = tmm.GEMM_F32, tmm.GEMM_F16, tmm.GEMM_BF16, tmm.GEMM_E4M3, tmm.GEMM_E2M1
OK, V, U, AL, NH = (tmm.GEMM_OK, tmm.GEMM_ERR_INVALID_VALUE, tmm.GEMM_ERR_UNSUPPORTED,
                    tmm.GEMM_ERR_ALIAS, tmm.GEMM_ERR_INVALID_HANDLE)
BIAS, GELU = tmm.GEMM_EPI_BIAS, tmm.GEMM_EPI_GELU
# Fake, well-separated device addresses: the checks never dereference them.
PA, PB, PC, PD, PE, PF, PG, PH = (0x1000000000 * i for i in range(1, 9))


def test_symbols_are_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "gemm_experts.h")).read()
    syms = sorted(set(re.findall(r"GEMM_API\s+[\w\s\*]*?\b(gemm_\w+)\s*\(", text)))
    assert sorted(tmm.EXPERTS_EXPORTS) == syms
    for s in syms:
        assert hasattr(tmm.library(), s) and hasattr(tmm, s)
    for name, v in re.findall(r"\b(GEMM_SCORE_\w+) = (\d+)", text):
        assert getattr(tmm, name) == int(v)


def route(T=100, E=64, k=4, x=PA, ldl=None, t=F32, score=1, bias=None, groups=1, best=1, of=1, renorm=0,
          expert=PB, weight=PC, place=PD, offsets=PE, ws=PF, nb=None):
    if nb is None:
        nb = max(0, tmm.gemm_route_workspace_bytes(T, E))
    return tmm.gemm_check_args_route(T, E, k, x, E if ldl is None else ldl, t, score, bias, groups, best, of,
                                     renorm, expert, weight, place, offsets, ws, nb)


def test_route():
    for t in (F32, F16, BF16):
        for score in (0, 1):
            assert route(t=t, score=score) == OK and route(t=t, score=score, bias=PG, renorm=1) == OK
    assert route(t=E4M3) == U and route(score=2) == V and route(score=-1) == V and route(renorm=2) == V
    assert route(T=-1) == V and route(E=0, k=1) == V and route(k=0) == V and route(k=65) == V
    assert route(k=33) == U and route(k=32) == OK
    assert route(E=1024) == OK and route(E=1025) == U and route(E=1, k=1) == OK
    assert route(T=2 ** 29, E=2, k=2, nb=2 ** 40) == OK and route(T=2 ** 29 + 1, E=2, k=2, nb=2 ** 40) == U
    assert route(T=2 ** 29, E=4, k=4, nb=2 ** 40) == U                 # pairs past 31 bits
    assert route(ldl=63) == V
    for name in ("x", "expert", "weight", "place", "offsets", "ws"):
        assert route(**{name: None}) == V, name
    assert route(offsets=PE + 4) == V
    # groups
    assert route(groups=8, best=2, of=2) == OK and route(groups=8, best=8, of=1) == OK
    assert route(groups=3) == V and route(groups=0) == V and route(groups=8, best=0) == V
    assert route(groups=8, best=9) == V and route(groups=8, best=4, of=3) == V and route(of=0) == V
    assert route(groups=64, best=4) == OK and route(groups=64, best=3) == V      # 3 experts for 4 slots
    assert route(E=128, groups=128, best=4) == U
    # workspace
    need = tmm.gemm_route_workspace_bytes(100, 64)
    assert need > 0 and route(nb=need - 1) == V and route(nb=need) == OK and route(nb=-1) == V
    assert route(ws=PF + 8) == V
    assert tmm.gemm_route_workspace_bytes(64, 64) == 0 and route(T=64, ws=None, nb=0) == OK
    assert tmm.gemm_route_workspace_bytes(-1, 4) == V and tmm.gemm_route_workspace_bytes(4, 0) == V
    assert tmm.gemm_route_workspace_bytes(4, 1025) == U and tmm.gemm_route_workspace_bytes(2 ** 30, 4) == U
    # no tokens: only the offsets
    assert route(T=0, x=None, expert=None, weight=None, place=None, ws=None) == OK
    assert route(T=0, offsets=None) == V
    # results against what is read and against each other
    size = 100 * 4 * 4
    assert route(expert=PA) == AL and route(weight=PA + 100 * 64 * 4 - 4) == AL
    assert route(weight=PA + 100 * 64 * 4) == OK
    assert route(place=PB + size - 4) == AL and route(place=PB + size) == OK
    assert route(bias=PE + 64 * 8) == AL and route(bias=PE + 65 * 8) == OK
    assert route(ws=PB) == AL and route(ws=PA) == AL and route(offsets=PC) == AL
    with pytest.raises(tmm.GemmError):
        tmm.route_workspace_bytes(4, 1025)


def grad(T=100, E=64, k=4, x=PA, ldl=None, t=F32, score=0, renorm=0, expert=PB, dw=PC, dx=PD, ldd=None):
    return tmm.gemm_check_args_route_grad(T, E, k, x, E if ldl is None else ldl, t, score, renorm, expert, dw,
                                          dx, E if ldd is None else ldd)


def test_route_grad():
    for t in (F32, F16, BF16):
        assert grad(t=t) == OK
    assert grad(t=E4M3) == U and grad(score=3) == V and grad(renorm=-1) == V and grad(k=0) == V
    assert grad(T=-1) == V and grad(k=65) == V and grad(k=33) == U and grad(E=1025) == U
    assert grad(ldl=63) == V and grad(ldd=63) == V
    for name in ("x", "expert", "dw", "dx"):
        assert grad(**{name: None}) == V, name
    assert grad(T=0, x=None, expert=None, dw=None, dx=None) == OK
    assert grad(dx=PA) == AL and grad(dx=PB) == AL and grad(dx=PC + 1599) == AL and grad(dx=PC + 1600) == OK


def move(call, T=40, k=2, K=64, X=PA, ldx=None, t=BF16, place=PB, R=80, w=PC, A=PD, lda=None, D=PE, dw=PF):
    ldx, lda = K if ldx is None else ldx, K if lda is None else lda
    if call == "dispatch":
        return tmm.gemm_check_args_dispatch_rows(T, k, K, X, ldx, t, place, R, A, lda)
    if call == "combine":
        return tmm.gemm_check_args_combine_rows(T, k, K, X, ldx, t, place, R, w, A, lda)
    return tmm.gemm_check_args_combine_rows_grad(T, k, K, D, K, X, ldx, t, place, R, w, A, lda, dw)


@pytest.mark.parametrize("call", ["dispatch", "combine", "grad"])
def test_moves(call):
    for t in (F32, F16, BF16):
        assert move(call, t=t) == OK
    assert move(call, t=E4M3) == U and move(call, T=-1) == V and move(call, k=0) == V
    assert move(call, K=-1, ldx=0, lda=0) == V and move(call, R=-1) == V
    assert move(call, T=2 ** 30, k=2) == U and move(call, R=2 ** 31) == U
    assert move(call, ldx=63) == V and move(call, lda=63) == V
    assert move(call, X=None) == V and move(call, A=None) == V and move(call, place=None) == V
    assert move(call, T=0, X=None, A=None, place=None, D=None, dw=None) == OK
    assert move(call, A=PA) == AL and move(call, A=PB) == AL and move(call, A=PB + 320) == OK


def test_moves_each():
    assert move("dispatch", R=0, X=None, A=None) == OK and move("dispatch", K=0, X=None, A=None) == OK
    assert move("combine", w=None) == OK and move("combine", R=0, X=None) == OK
    assert move("combine", A=PC + 300) == AL and move("combine", A=PC + 320) == OK
    assert move("grad", w=None) == V and move("grad", dw=None) == V and move("grad", D=None) == V
    assert move("grad", K=0, X=None, A=None, D=None) == OK and move("grad", R=0, X=None, A=None) == OK
    assert move("grad", dw=PC) == AL and move("grad", dw=PD) == AL and move("grad", D=PD) == AL
    assert move("grad", dw=PA + 80 * 128 - 4) == AL and move("grad", dw=PA + 80 * 128) == OK


def quant(M=40, K=64, X=PA, ldx=None, t=BF16, top=1, place=None, R=None, Q=PB, ldq=None, qt=E2M1, S=PC,
          lds=None):
    return tmm.gemm_check_args_quantize_mx(M, K, X, K if ldx is None else ldx, t, top, place,
                                           M if R is None else R, Q, K if ldq is None else ldq, qt, S,
                                           K // 32 if lds is None else lds)


def test_quantize_mx():
    for t in (F32, F16, BF16):
        assert quant(t=t) == OK and quant(t=t, top=3, place=PD, R=120) == OK
    assert quant(t=E4M3) == U and quant(qt=E4M3) == U and quant(M=2 ** 31) == U
    assert quant(M=-1) == V and quant(K=48) == V and quant(K=-32, ldx=0, ldq=0, lds=0) == V
    assert quant(top=2) == V and quant(R=41) == V and quant(top=0, place=PD) == V
    assert quant(X=None) == V and quant(Q=None) == V and quant(S=None) == V
    assert quant(ldx=63) == V and quant(ldq=63) == V and quant(ldq=65) == V and quant(lds=1) == V
    assert quant(M=0, X=None, Q=None, S=None) == OK and quant(K=0, X=None, Q=None, S=None) == OK
    assert quant(R=0, place=PD, Q=None, S=None) == OK
    assert quant(Q=PA + 40 * 128 - 1) == AL and quant(Q=PA + 40 * 128) == OK
    assert quant(S=PB + 40 * 32 - 1) == AL and quant(S=PB + 40 * 32) == OK and quant(S=PA) == AL
    assert quant(place=PB, top=1, R=40) == AL


def mx(G=3, off=PA, M=40, N=48, K=64, A=PB, lda=None, sa=PC, ldsa=None, B=PD, ldb=None, stride=None, sb=PE,
       ldsb=None, stride_sb=None, C=PF, ldc=None, t=E2M1, ct=BF16, epi=0, bias=None):
    ldb = K if ldb is None else ldb
    ldsb = max(K, 0) // 32 if ldsb is None else ldsb
    return tmm.gemm_check_args_grouped_mx(
        G, off, M, N, K, A, K if lda is None else lda, sa, max(K, 0) // 32 if ldsa is None else ldsa, B, ldb,
        N * ldb if stride is None else stride, sb, ldsb, N * ldsb if stride_sb is None else stride_sb, C,
        N if ldc is None else ldc, t, ct, epi, bias)


def test_grouped_mx():
    for ct in (F32, F16, BF16):
        assert mx(ct=ct) == OK and mx(ct=ct, epi=BIAS | GELU, bias=PG) == OK
    assert mx(t=E4M3) == U and mx(ct=E4M3) == U and mx(t=BF16) == U
    assert mx(M=-1) == V and mx(N=-1) == V and mx(K=-32) == V and mx(G=-1) == V and mx(epi=4) == V
    assert mx(K=48, ldsa=2, ldsb=2) == V
    assert mx(off=None) == V and mx(off=None, G=1) == OK and mx(off=PA + 4) == V
    for name in ("A", "B", "C", "sa", "sb"):
        assert mx(**{name: None}) == V, name
    assert mx(lda=62) == V and mx(lda=65) == V and mx(ldb=62) == V and mx(ldb=65) == V and mx(ldc=47) == V
    assert mx(ldsa=1) == V and mx(ldsb=1) == V
    assert mx(stride=-2) == V and mx(stride=3) == V and mx(stride_sb=-1) == V
    assert mx(stride=0, stride_sb=0) == OK and mx(epi=BIAS) == V
    assert mx(G=65535, stride=0, stride_sb=0) == OK and mx(G=65536, stride=0, stride_sb=0) == U
    assert mx(M=2 ** 31) == U and mx(N=2 ** 31) == U and mx(M=2 ** 30, N=2 ** 30) == U
    assert mx(M=0, A=None, C=None, off=None) == OK and mx(N=0, C=None) == OK and mx(G=0, off=None) == OK
    assert mx(K=0, A=None, B=None, sa=None, sb=None) == OK
    size = 40 * 48 * 2
    assert mx(C=PB) == AL and mx(C=PB + 40 * 32 - 1) == AL and mx(C=PB + 40 * 32) == OK
    assert mx(C=PC + 79) == AL and mx(C=PC + 80) == OK
    assert mx(C=PD + 3 * 48 * 32 - 1) == AL and mx(C=PD + 3 * 48 * 32) == OK
    assert mx(C=PE + 3 * 48 * 2 - 1) == AL and mx(C=PE + 3 * 48 * 2) == OK
    assert mx(C=PA + 31) == AL and mx(C=PA + 32) == OK
    assert mx(epi=BIAS, bias=PF + size - 4) == AL and mx(epi=BIAS, bias=PF + size) == OK


def test_null_handle():
    assert tmm.gemm_route(None, None, 4, 4, 1, PA, 4, F32, 0, None, 1, 1, 1, 0, 1.0, PB, PC, PD, PE, None, 0) == NH
    assert tmm.gemm_route_grad(None, None, 4, 4, 1, PA, 4, F32, 0, 0, 1.0, PB, PC, PD, 4) == NH
    assert tmm.gemm_dispatch_rows(None, None, 4, 1, 4, PA, 4, F32, PB, 4, PC, 4) == NH
    assert tmm.gemm_combine_rows(None, None, 4, 1, 4, PA, 4, F32, PB, 4, None, 0.0, PC, 4) == NH
    assert tmm.gemm_combine_rows_grad(None, None, 4, 1, 4, PA, 4, PB, 4, F32, PC, 4, PD, PE, 4, PF) == NH
    assert tmm.gemm_quantize_mx(None, None, 4, 32, PA, 32, F32, 1, None, 4, PB, 32, E2M1, PC, 1) == NH
    assert tmm.gemm_run_grouped_mx(None, 0, None, 1, PA, 4, 4, 32, 1.0, PB, 32, PC, 1, PD, 32, 128, PE, 1, 4,
                                   0.0, PF, 4, E2M1, BF16, 0, None) == NH
