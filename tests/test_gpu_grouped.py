"""Products grouped by expert, their gradients, 8-bit integer products and row quantization on the
GPU, against plain numpy in 64 bits.

Tolerances (fixed before the first run): a product's error is measured against D = sum |a b| (plus
|beta C| and |bias|), as the parity gate does: fp32 sums in any order stay within K 2^-23 of it,
the epilogue adds 4 (16 more with GELU) fp32 roundings, and the result is rounded once, by half a
step of its type relative to the value.  An integer sum is exact, so only the roundings of its
scaling (4) and of the epilogue count.  Codes and NaN have to be equal.
"""
import numpy as np
import pytest
from scipy.special import erfc

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tiled_matrix_multiply_amd as tmm
    h = tmm.Gemm(0)
    yield h
    h.close()


def T():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")
    return t if dtype is None else t.to(T()[dtype])


def host(t):
    return t.double().cpu().numpy()


def effective(offsets, M):
    """The offsets as the kernels read them: clamped to 0 .. M, raised to the largest before."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, M))


def gelu(x):
    with np.errstate(invalid="ignore"):
        return 0.5 * x * erfc(-x / np.sqrt(2.0))


def check(got, ref, denom, tol, c_type, what):
    """|got - ref| <= tol * max(denom, |ref|), and infinities and NaN where the reference has them."""
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), what
    err = np.abs(got[fin] - ref[fin]) - TINY[c_type]
    lim = tol * np.maximum(denom[fin], np.abs(ref[fin]))
    bad = ~(err <= lim)
    assert not bad.any(), (what, int(bad.sum()), float((err - lim).max()))


def epilogue(v, D, beta, cin, bias, do_gelu):
    if beta:
        v, D = v + beta * cin, D + np.abs(beta * cin)
    if bias is not None:
        v, D = v + bias, D + np.abs(bias)
    return (gelu(v) if do_gelu else v), D


def offsets_of(sizes, start=0):
    return np.concatenate([[start], start + np.cumsum(sizes)]).astype(np.int64)


RNG = np.random.default_rng
MANY = [0, 3, 1, 0, 17] * 14 + [33]  # 71 groups: more than a wave has lanes
SIZES = [[0], [1], [5, 0, 7], [0, 0, 3, 0], [64, 65, 1, 0, 127], [300, 2, 513], MANY]
DIMS = [(1, 1), (33, 17), (64, 64), (100, 72), (264, 136), (136, 1000)]

ANY = 1
KERNELS = [ANY]


def run_grouped(g, sizes, N, K, *, trans_b, t, kernel=0, alpha=1.0, beta=0.0, bias=False,
                do_gelu=False, lda=None, ldb=None, ldc=None, stride=None, offsets=None, M=None,
                seed=0, poison=None, stream=None):
    """One call against the plain form; `poison` fills what must not be read or written."""
    import torch
    G = len(sizes)
    off = offsets_of(sizes) if offsets is None else np.asarray(offsets, dtype=np.int64)
    M = int(off[-1]) if M is None else M
    eff = effective(off, M)
    rng = RNG(seed)
    lda, ldc = lda or K, ldc or N
    brows, bcols = (N, K) if trans_b else (K, N)
    ldb = ldb or bcols
    stride = brows * ldb if stride is None else stride
    fill = 0.0 if poison is None else poison
    A = np.full((M, lda), fill)
    A[:, :K] = rng.standard_normal((M, K))
    inside = np.zeros(M, dtype=bool)
    for q in range(G):
        inside[eff[q]:eff[q + 1]] = True
    if poison is not None:
        A[~inside] = poison
    B = np.full(max(1, (G - 1) * stride + brows * ldb), fill)
    for q in range(G):
        view = B[q * stride:q * stride + brows * ldb].reshape(brows, ldb)
        view[:, :bcols] = rng.standard_normal((brows, bcols)) * max(K, 1) ** -0.5
    C = rng.standard_normal((M, ldc))
    bias_h = 0.5 * rng.standard_normal((G, N)).astype(np.float32) if bias else None
    dA, dB, dC = dev(A, t), dev(B, t), dev(C, t)
    before = dC.clone()
    import tiled_matrix_multiply_amd as tmm
    g.run_grouped(dA, dB, dC, dev(off), groups=G, M=M, N=N, K=K, trans_b=trans_b, a_type=t,
                  alpha=alpha, beta=beta,
                  epilogue=(tmm.GEMM_EPI_BIAS if bias else 0) | (tmm.GEMM_EPI_GELU if do_gelu else 0),
                  bias=dev(bias_h) if bias else None, lda=lda, ldb=ldb, stride_b=stride, ldc=ldc,
                  kernel=kernel, stream=stream)
    torch.cuda.synchronize()
    A64, B64, C64, got = host(dA), host(dB), host(before), host(dC)
    ref, D = C64[:, :N].copy(), np.zeros((M, N))
    for q in range(G):
        rows = slice(eff[q], eff[q + 1])
        b = B64[q * stride:q * stride + brows * ldb].reshape(brows, ldb)[:, :bcols]
        b = b.T if trans_b else b
        a = A64[rows, :K]
        ref[rows], D[rows] = epilogue(alpha * (a @ b), abs(alpha) * (np.abs(a) @ np.abs(b)), beta,
                                      C64[rows, :N], bias_h[q].astype(np.float64) if bias else None,
                                      do_gelu)
    tol = K * 2.0 ** -23 + HALF_STEP[t] + (20 if do_gelu else 4) * U32
    check(got[:, :N], ref, D, tol, t, (sizes, N, K, trans_b, t, kernel))
    same = torch.equal(dC[:, N:].view(torch.int16), before[:, N:].view(torch.int16))
    assert same, "columns past N"
    out = torch.from_numpy(~inside).to(dC.device)
    assert torch.equal(dC[out].view(torch.int16), before[out].view(torch.int16)), "rows of no group"
    return dC


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_grouped_sizes(g, t, trans_b, kernel):
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(DIMS):
            if kernel > ANY:
                N, K = -(-N // 8) * 8, -(-K // 8) * 8
            print(f"[grouped] {t} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_grouped(g, sizes, N, K, trans_b=trans_b, t=t, kernel=kernel, seed=10 * i + j,
                        bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                        alpha=0.75 if j % 2 else 1.0, beta=-0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("trans_b", [False, True])
def test_grouped_strides_and_rows_of_no_group(g, trans_b, kernel):
    """Padded rows and matrices, rows before the first and past the last group, and NaN or the
    type's infinities in everything that belongs to no operand: none of it comes through."""
    for poison in (np.nan, np.inf):
        run_grouped(g, [40, 0, 90], 72, 104, trans_b=trans_b, t="bf16", kernel=kernel, lda=128,
                    ldb=120, ldc=80, stride=120 * 112, offsets=[7, 47, 47, 137], M=150,
                    poison=poison, bias=True, seed=3)
    run_grouped(g, [40, 9, 90], 72, 104, trans_b=trans_b, t="f16", kernel=kernel, stride=0, seed=4)


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("offsets", [[0, 50, 20, 100], [-5, 30, 300, 80], [90, 10, 20, 30],
                                     [2 ** 40, 0, 5, 9], [-2 ** 62, 2 ** 62, 3, 2 ** 62]])
def test_grouped_offsets_out_of_order(g, offsets, kernel):
    """Offsets that fall or leave the matrix are clamped and raised: every group stays inside."""
    run_grouped(g, [0, 0, 0], 64, 64, trans_b=True, t="bf16", kernel=kernel, offsets=offsets, M=100,
                seed=5)


def test_grouped_misaligned_pointers(g):
    """Operands that start in the middle of 16 bytes."""
    import torch
    for t in ("bf16", "f16"):
        A = torch.randn(71, 64, device="cuda").to(T()[t]).flatten()
        B = torch.randn(2 * 64 * 40 + 1, device="cuda").to(T()[t])
        C = torch.zeros(71 * 40 + 3, device="cuda", dtype=T()[t])
        off = dev(np.array([0, 30, 70], dtype=np.int64))
        g.run_grouped(A[1:], B[1:], C[3:], off, groups=2, M=70, N=40, K=64, a_type=t)
        a, b = host(A[1:1 + 70 * 64]).reshape(70, 64), host(B[1:]).reshape(2, 64, 40)
        ref = np.concatenate([a[:30] @ b[0], a[30:] @ b[1]])
        D = np.concatenate([abs(a[:30]) @ abs(b[0]), abs(a[30:]) @ abs(b[1])])
        check(host(C[3:3 + 2800]).reshape(70, 40), ref, D, 64 * 2.0 ** -23 + HALF_STEP[t] + 4 * U32, t, t)
        assert not C[:3].any() and not C[2803:].any()


@pytest.mark.parametrize("kernel", [0] + KERNELS)
def test_grouped_infinities_stay_in_their_rows(g, kernel):
    import torch
    A = torch.randn(96, 64, device="cuda").to(torch.bfloat16)
    A[10, 3], A[50, 60], A[70, 0] = float("inf"), float("nan"), float("-inf")
    B = torch.randn(3, 64, 64, device="cuda").to(torch.bfloat16)
    C = torch.zeros(96, 64, device="cuda", dtype=torch.bfloat16)
    g.run_grouped(A, B, C, dev(np.array([0, 32, 64, 96], dtype=np.int64)), groups=3, M=96, N=64,
                  K=64, kernel=kernel)
    bad = ~torch.isfinite(C).all(dim=1)
    assert sorted(torch.nonzero(bad).flatten().tolist()) == [10, 50, 70]
    assert torch.isnan(C[50]).all()


@pytest.mark.parametrize("kernel", [0] + KERNELS)
def test_grouped_far_addresses(g, kernel):
    """Rows of A and C and matrices of B further than 2^32 bytes from the start."""
    import torch
    M, lda, ldc, N, K, G = 150000, 16384, 16384, 64, 128, 3
    A = torch.zeros(M, lda, device="cuda", dtype=torch.bfloat16)
    C = torch.zeros(M, ldc, device="cuda", dtype=torch.bfloat16)
    stride = 3 << 29
    B = torch.empty(2 * stride + N * K, device="cuda", dtype=torch.bfloat16)
    off = [M - 100, M - 60, M - 60, M]
    A[M - 100:, :K] = torch.randn(100, K, device="cuda").to(torch.bfloat16)
    ref, D = [], []
    for q in range(G):
        b = torch.randn(N, K, device="cuda").to(torch.bfloat16)
        B[q * stride:q * stride + N * K] = b.flatten()
        a = host(A[off[q]:off[q + 1], :K])
        ref.append(a @ host(b).T)
        D.append(np.abs(a) @ np.abs(host(b)).T)
    g.run_grouped(A, B, C, dev(np.array(off, dtype=np.int64)), groups=G, M=M, N=N, K=K, trans_b=True,
                  lda=lda, ldc=ldc, stride_b=stride, kernel=kernel)
    check(host(C[M - 100:, :N]), np.concatenate(ref), np.concatenate(D),
          K * 2.0 ** -23 + HALF_STEP["bf16"] + 4 * U32, "bf16", "far")
    assert not C[:M - 100].any() and not C[:, N:].any()


# ---------------------------------------------------------------------- weight gradient --

def run_wgrad(g, sizes, N, K, *, trans_b, t, ct, kernel=0, alpha=1.0, beta=0.0, dbias=True, seed=0,
              lda=None, ldd=None, ldc=None, stride=None, offsets=None, M=None, poison=None):
    import torch
    G = len(sizes)
    off = offsets_of(sizes) if offsets is None else np.asarray(offsets, dtype=np.int64)
    M = int(off[-1]) if M is None else M
    eff = effective(off, M)
    rng = RNG(seed)
    rows, cols = (N, K) if trans_b else (K, N)
    lda, ldd, ldc = lda or K, ldd or N, ldc or cols
    stride = rows * ldc if stride is None else stride
    A, Dm = rng.standard_normal((M, lda)), rng.standard_normal((M, ldd))
    if poison is not None:
        keep = np.zeros(M, dtype=bool)
        for q in range(G):
            keep[eff[q]:eff[q + 1]] = True
        A[:, K:], Dm[:, N:], A[~keep], Dm[~keep] = poison, poison, poison, poison
    C = rng.standard_normal((G - 1) * stride + rows * ldc)
    dA, dD, dC = dev(A, t), dev(Dm, t), dev(C, ct)
    before = dC.clone()
    db = torch.full((G, N), float("nan"), device="cuda") if dbias else None
    g.run_grouped_wgrad(dA, dD, dC, dev(off), groups=G, M=M, N=N, K=K, trans_b=trans_b, a_type=t,
                        c_type=ct, alpha=alpha, beta=beta, dbias=db, lda=lda, ldd=ldd, ldc=ldc,
                        stride_c=stride, kernel=kernel)
    torch.cuda.synchronize()
    A64, D64, C64, got = host(dA), host(dD), host(before), host(dC)
    touched = np.zeros(C.size, dtype=bool)
    for q in range(G):
        r = slice(eff[q], eff[q + 1])
        a, d = A64[r, :K], D64[r, :N]
        w, den = a.T @ d, np.abs(a).T @ np.abs(d)
        if trans_b:
            w, den = w.T, den.T
        cut = slice(q * stride, q * stride + rows * ldc)
        cin = C64[cut].reshape(rows, ldc)[:, :cols]
        ref, den = epilogue(alpha * w, abs(alpha) * den, beta, cin, None, False)
        n = int(eff[q + 1] - eff[q])
        check(got[cut].reshape(rows, ldc)[:, :cols], ref, den, n * 2.0 ** -23 + HALF_STEP[ct] + 4 * U32, ct,
              ("wgrad", sizes, N, K, trans_b, q))
        touched[cut].reshape(rows, ldc)[:, :cols] = True
        if dbias:
            check(host(db[q]), d.sum(0), np.abs(d).sum(0), (n + 2) * U32, "f32", ("dbias", sizes, q))
    idle = torch.from_numpy(~touched).cuda()
    iv = torch.int32 if ct == "f32" else torch.int16
    assert torch.equal(dC[idle].view(iv), before[idle].view(iv))


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_wgrad_sizes(g, t, ct, trans_b, kernel):
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(DIMS[:5]):
            if kernel > ANY:
                N, K = -(-N // 8) * 8, -(-K // 8) * 8
            print(f"[wgrad] {t} {ct} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_wgrad(g, sizes, N, K, trans_b=trans_b, t=t, ct=ct, kernel=kernel, seed=10 * i + j,
                      dbias=(i + j) % 3 != 0, alpha=0.5 if j % 2 else 1.0,
                      beta=1.0 if (i + j) % 2 else 0.0)


@pytest.mark.parametrize("kernel", [0] + KERNELS)
def test_wgrad_strides_and_rows_of_no_group(g, kernel):
    for poison in (np.nan, np.inf):
        run_wgrad(g, [40, 0, 90], 72, 104, trans_b=False, t="bf16", ct="f32", kernel=kernel, lda=128,
                  ldd=80, ldc=84, stride=84 * 110, offsets=[7, 47, 47, 137], M=150, poison=poison)


def test_wgrad_bad_offsets_and_no_rows(g):
    run_wgrad(g, [0, 0, 0], 64, 64, trans_b=True, t="bf16", ct="bf16", offsets=[0, 50, 20, 900], M=100)
    run_wgrad(g, [0, 0], 64, 40, trans_b=True, t="bf16", ct="bf16", beta=0.5)      # M = 0
    run_wgrad(g, [0, 0], 64, 40, trans_b=False, t="f16", ct="f32")


def test_gradients_against_differences(g):
    """The call's gradients of f = sum(W * forward(A, B, bias)) against central differences of the
    plain forward in 64 bits along random directions (f is linear in each, so the difference
    quotient has no truncation error)."""
    import torch
    rng = RNG(7)
    sizes, N, K, t = [9, 0, 20], 24, 40, "f16"
    off = offsets_of(sizes)
    A = dev(rng.standard_normal((29, K)), t)
    B = dev(rng.standard_normal((3, N, K)), t)
    W = dev(rng.standard_normal((29, N)), t)
    bias = rng.standard_normal((3, N))
    dA, dB = torch.zeros_like(A), torch.zeros(3, N, K, device="cuda")
    db = torch.zeros(3, N, device="cuda")
    o = dev(off)
    g.run_grouped(W, B, dA, o, groups=3, M=29, N=K, K=N, trans_b=False, a_type=t)
    g.run_grouped_wgrad(A, W, dB, o, groups=3, M=29, N=N, K=K, trans_b=True, a_type=t, c_type="f32",
                        dbias=db)
    torch.cuda.synchronize()
    A64, B64, W64 = host(A), host(B), host(W)

    def f(a, b, c):
        return sum((W64[off[q]:off[q + 1]] * (a[off[q]:off[q + 1]] @ b[q].T + c[q])).sum() for q in range(3))

    for grad, x in ((dA, 0), (dB, 1), (db, 2)):
        args = [A64, B64, bias]
        E = rng.standard_normal(args[x].shape)
        up, down = list(args), list(args)
        up[x], down[x] = args[x] + E, args[x] - E
        want = (f(*up) - f(*down)) / 2
        got = (host(grad) * E).sum()
        # each entry of the gradient is off by half a step of its type and the fp32 sum's error
        # relative to sum |.|, at most 29 terms
        half = HALF_STEP["f16"] if x == 0 else U32
        def size(q):
            a, w, e = (np.abs(v[off[q]:off[q + 1]]) for v in (A64, W64, E)) if x == 0 else \
                (np.abs(A64[off[q]:off[q + 1]]), np.abs(W64[off[q]:off[q + 1]]), np.abs(E[q]))
            return {0: lambda: (w @ np.abs(B64[q]) * e).sum(), 1: lambda: (w.T @ a * e).sum(),
                    2: lambda: (w.sum(0) * e).sum()}[x]()

        scale = sum(size(q) for q in range(3))
        assert abs(got - want) <= (half + 40 * 2.0 ** -23) * scale + 1e-9


# ----------------------------------------------------------------- 8-bit integers --

def run_i8(g, sizes, N, K, *, trans_b, ct, grouped=True, kernel=0, alpha=1.0, beta=0.0, bias=False,
           do_gelu=False, seed=0, lda=None, ldb=None, ldc=None, lo=-128, hi=127):
    import torch
    import tiled_matrix_multiply_amd as tmm
    G = len(sizes)
    off = offsets_of(sizes)
    M = int(off[-1])
    rng = RNG(seed)
    brows, bcols = (N, K) if trans_b else (K, N)
    lda, ldb, ldc = lda or K, ldb or bcols, ldc or N
    A = rng.integers(lo, hi, (M, lda), endpoint=True).astype(np.int8)
    B = rng.integers(lo, hi, (G, brows, ldb), endpoint=True).astype(np.int8)
    sa = rng.uniform(0.001, 0.1, M).astype(np.float32)
    sb = rng.uniform(0.001, 0.01, (G, N)).astype(np.float32)
    bias_h = rng.standard_normal((G, N)).astype(np.float32) if bias else None
    C = dev(rng.standard_normal((M, ldc)), ct)
    before = host(C)
    kw = dict(M=M, N=N, K=K, trans_b=trans_b, c_type=ct, alpha=alpha, beta=beta, lda=lda, ldb=ldb, ldc=ldc,
              epilogue=(tmm.GEMM_EPI_BIAS if bias else 0) | (tmm.GEMM_EPI_GELU if do_gelu else 0),
              bias=dev(bias_h) if bias else None, kernel=kernel)
    if grouped:
        g.run_grouped_i8(dev(A), dev(sa), dev(B), dev(sb), C, dev(off), groups=G, **kw)
    else:
        g.run_i8(dev(A), dev(sa), dev(B), dev(sb), C, **kw)
    torch.cuda.synchronize()
    ref, D = np.zeros((M, N)), np.zeros((M, N))
    for q in range(G):
        r = slice(off[q], off[q + 1])
        b = B[q][:, :bcols].astype(np.int64)
        s = A[r, :K].astype(np.int64) @ (b.T if trans_b else b)
        v = alpha * s * sa[r].astype(np.float64)[:, None] * sb[q].astype(np.float64)
        ref[r], D[r] = epilogue(v, np.abs(v), beta, before[r, :N],
                                bias_h[q].astype(np.float64) if bias else None, do_gelu)
    got = host(C)
    tol = HALF_STEP[ct] + (4 + (20 if do_gelu else 4)) * U32
    check(got[:, :N], ref, D, tol, ct, ("i8", sizes, N, K, trans_b, ct, kernel))
    assert np.array_equal(got[:, N:], before[:, N:])


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("trans_b", [False, True])
@pytest.mark.parametrize("ct", ["bf16", "f16", "f32"])
def test_i8_sizes(g, ct, trans_b, kernel):
    for i, sizes in enumerate(SIZES):
        for j, (N, K) in enumerate(DIMS):
            if kernel > ANY:
                N, K = -(-N // 16) * 16, -(-K // 16) * 16
            print(f"[i8] {ct} {trans_b} {kernel} {sizes[:6]} {N} {K}", flush=True)
            run_i8(g, sizes, N, K, trans_b=trans_b, ct=ct, grouped=len(sizes) > 1 or j % 2 == 0,
                   kernel=kernel, seed=10 * i + j, bias=(i + j) % 2 == 0, do_gelu=(i + j) % 3 == 0,
                   alpha=-0.75 if j % 2 else 1.0, beta=0.5 if (i + j) % 4 == 1 else 0.0)


@pytest.mark.parametrize("kernel", [0] + KERNELS)
@pytest.mark.parametrize("trans_b", [False, True])
def test_i8_exact_sums(g, trans_b, kernel):
    """Sums past 24 bits, at the ends of the codes' range: the integer sum loses nothing.  With
    scales of 1 an fp32 result is the sum rounded once."""
    import torch
    M, N, K = 5, 32, 8192 + 16
    A = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    A[1] = 127
    A[2:] = torch.randint(-128, 128, (3, K), device="cuda").to(torch.int8)
    B = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    B[8:16] = 127
    B[16:] = torch.randint(-128, 128, (16, K), device="cuda").to(torch.int8)
    C = torch.zeros(M, N, device="cuda")
    one = torch.ones(64, device="cuda")
    Bs = B if trans_b else B.t().contiguous()
    g.run_i8(A, one, Bs, one, C, M=M, N=N, K=K, trans_b=trans_b, c_type="f32", kernel=kernel)
    want = (A.cpu().long() @ B.cpu().long().t()).float()
    assert torch.equal(C.cpu(), want)


@pytest.mark.parametrize("kernel", [0] + KERNELS)
def test_i8_longest_sum(g, kernel):
    """K = 131071 at -128 x -128: the largest sum 31 bits hold."""
    import torch
    K = 131071
    lda = 131072
    A = torch.full((2, lda), -128, dtype=torch.int8, device="cuda")
    B = torch.full((16, lda), -128, dtype=torch.int8, device="cuda")
    C = torch.zeros(2, 16, device="cuda")
    one = torch.ones(16, device="cuda")
    g.run_i8(A, one, B, one, C, M=2, N=16, K=K, lda=lda, ldb=lda, trans_b=True, c_type="f32",
             kernel=kernel)
    assert (C.cpu().double() == float(np.float32(K * 128 * 128))).all()


@pytest.mark.parametrize("kernel", [0] + KERNELS)
def test_i8_bad_scale_stays_in_its_row(g, kernel):
    import torch
    A = torch.randint(-127, 128, (70, 64), device="cuda").to(torch.int8)
    B = torch.randint(-127, 128, (48, 64), device="cuda").to(torch.int8)
    sa, sb = torch.rand(70, device="cuda") + 0.1, torch.rand(48, device="cuda") + 0.1
    sa[3], sb[40] = float("nan"), 0.0
    C = torch.zeros(70, 48, device="cuda")
    g.run_i8(A, sa, B, sb, C, M=70, N=48, K=64, trans_b=True, c_type="f32", kernel=kernel)
    bad = torch.isnan(C)
    assert bad[3].all() and not bad[:3].any() and not bad[4:].any()
    assert (C[4:, 40] == 0).all()


# ------------------------------------------------------------------- row quantization --

def quantize(x):
    """Codes and scales of float64 rows by the definition (scale rounded to fp32)."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = np.abs(x).max(axis=1, initial=0.0)
        s = (m / 127).astype(np.float32)
        live = (s > 0) & np.isfinite(s)
        q = np.where(live[:, None], np.rint(x / np.where(live, s, 1).astype(np.float64)[:, None]), 0)
    return np.clip(np.nan_to_num(q), -127, 127).astype(np.int8), s


def run_quantize(g, x, t, ldx=None, ldq=None, skew=0):
    """x: numpy values; the call's codes and scales have to equal the definition's."""
    import torch
    M, K = x.shape
    ldx, ldq = ldx or K, ldq or K
    X = torch.full((M * ldx + skew,), 1e4, device="cuda").to(T()[t])
    X[skew:].view(M, ldx)[:, :K] = dev(x, t) if x.dtype != np.float32 else dev(x)
    Q = torch.full((M, ldq), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    g.quantize_rows(X[skew:], Q, s, M=M, K=K, x_type=t, ldx=ldx, ldq=ldq)
    torch.cuda.synchronize()
    q, want = quantize(host(X[skew:].view(M, ldx)[:, :K]))
    assert np.array_equal(s.cpu().numpy(), want, equal_nan=True), (M, K, t)
    assert np.array_equal(Q[:, :K].cpu().numpy(), q), (M, K, t)
    assert (Q[:, K:] == 99).all()


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_quantize_sizes(g, t):
    rng = RNG(11)
    for M, K in [(1, 1), (1, 7), (3, 8), (2, 64), (5, 100), (1, 4096), (4, 1024), (70, 129), (3, 8192),
                 (2, 8200), (2, 20000), (300, 520), (1, 70001)]:
        print(f"[quantize] {t} {M} {K}", flush=True)
        run_quantize(g, rng.standard_normal((M, K)), t)
    run_quantize(g, rng.standard_normal((7, 100)), t, ldx=107, ldq=101)
    run_quantize(g, rng.standard_normal((7, 96)), t, ldx=112, ldq=128)
    run_quantize(g, rng.standard_normal((7, 96)), t, skew=3)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_quantize_ties_and_borders(g, t):
    """A row maximum of 127 * 2^e makes the scale a power of two and every half-integer a tie; others
    put values next to the borders."""
    rng = RNG(12)
    half = np.arange(-127, 127.5, 0.5)
    x = np.stack([np.resize(half, 600), np.resize(half * 2.0 ** -9, 600)])
    run_quantize(g, x, t)
    base = rng.uniform(1, 2, (40, 1))
    near = (rng.integers(-127, 127, (40, 500)) + 0.5) / 127 * base
    x = np.concatenate([base, near], axis=1)
    run_quantize(g, x.astype(np.float32) if t == "f32" else x, t)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_quantize_extremes(g, t):
    top = {"bf16": 3.3e38, "f16": 65504.0, "f32": 3.4e38}[t]
    low = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}[t]
    rng = RNG(13)
    x = rng.standard_normal((10, 256))
    x[0] = 0.0
    x[1] = low * rng.integers(-3, 4, 256)
    x[2] = np.clip(x[2], -1, 1) * top
    x[3, 7], x[4, 8], x[5, 9] = np.nan, np.inf, -np.inf
    x[6, 100] = np.nan
    x[6, 5] = np.inf
    x[7] = low * rng.integers(-200, 200, 256)
    x[8] = x[8] * (top * 2.0 ** -120)
    x[9] = -0.0
    run_quantize(g, x.astype(np.float32) if t == "f32" else x, t)


# ------------------------------------------------------------------- streams and graphs --

def test_streams_and_graph(g):
    """On a stream that is not the current one, and replayed from a graph with new offsets each
    time: the offsets are read when the kernels run."""
    import torch
    rng = RNG(14)
    M, N, K, G = 200, 64, 128, 4
    A = dev(rng.standard_normal((M, K)), "bf16")
    B = dev(rng.standard_normal((G, N, K)), "bf16")
    C = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    W = torch.zeros(G, N, K, device="cuda", dtype=torch.bfloat16)
    db = torch.zeros(G, N, device="cuda")
    Q, s = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    B8 = torch.randint(-127, 128, (G, N, K), device="cuda").to(torch.int8)
    sb = torch.rand(G, N, device="cuda")
    C8 = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    off = dev(np.array([0, 50, 60, 60, 200], dtype=np.int64))

    def call(stream=None):
        kw = dict(groups=G, M=M, N=N, K=K, trans_b=True, stream=stream)
        g.run_grouped(A, B, C, off, **kw)
        g.run_grouped_wgrad(A, C, W, off, dbias=db, **kw)
        g.quantize_rows(A, Q, s, M=M, K=K, stream=stream)
        g.run_grouped_i8(Q, s, B8, sb, C8, off, **kw)

    outs = (C, W, db, Q, s, C8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(side.cuda_stream)
    side.synchronize()
    first = [o.clone() for o in outs]
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cuts in ([0, 50, 60, 60, 200], [0, 0, 0, 0, 200], [0, 199, 199, 200, 200], [0, 10, 90, 150, 200]):
        off.copy_(torch.tensor(cuts))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replay = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replay, outs)), cuts


def test_repeated_calls_agree(g):
    """The same call twice gives the same bits: no sum depends on which wave comes first."""
    import torch
    A = torch.randn(3000, 512, device="cuda").to(torch.bfloat16)
    D = torch.randn(3000, 256, device="cuda").to(torch.bfloat16)
    off = dev(np.array([0, 1000, 1001, 3000], dtype=np.int64))
    outs = []
    for _ in range(3):
        C = torch.zeros(3, 256, 512, device="cuda")
        db = torch.zeros(3, 256, device="cuda")
        g.run_grouped_wgrad(A, D, C, off, groups=3, M=3000, N=256, K=512, trans_b=True, c_type="f32",
                            dbias=db)
        torch.cuda.synchronize()
        outs.append((C, db))
    for C, db in outs[1:]:
        assert torch.equal(C, outs[0][0]) and torch.equal(db, outs[0][1])
