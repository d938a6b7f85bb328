"""Paths of the grouped and 8-bit integer kernels that only larger calls take, against the formulas in
64 bits: the 256 x 256 tiles of the mixed kernel (kept whole, beside split ones, and with more small
tiles than workgroups that share them), the any-alignment tile whose K is not split, the streaming
kernel with 64 rows of a B stored K x N, and gradients whose tiles are dealt to the XCDs unevenly.
Copies of the rules that choose them say that each case takes its path.

Tolerances as test_gpu_grouped.py has them: K 2^-23 of sum |a b| for fp32 sums (none for integers), 4
fp32 roundings in the epilogue (16 more with GELU, 4 more for the scales), half a step of the result.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
U32 = 2.0 ** -24
AUTO, ANY, TILE_64, TILE_128, TILE_256, STREAM = range(6)


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tiled_matrix_multiply_amd as tmm
    h = tmm.Gemm(0)
    yield h
    h.close()


def dtype(t):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}[t]


def compute_units():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def ceil(a, b):
    return -(-a // b)


def check(got, ref, denom, tol, c_type, what):
    err = (got.double() - ref).abs() - TINY[c_type]
    over = err - tol * denom.maximum(ref.abs())
    assert bool(got.isfinite().all()) and float(over.max()) <= 0, (what, float(over.max()))


def product(g, sizes, N, K, *, nk, t, ct, kernel, grouped=True, pad=0, skew=0, bias=True, do_gelu=False, alpha=0.75,
            beta=0.0, seed=0):
    """One call: rows padded by `pad` elements that hold NaN (127 in 8 bits), and every operand `skew`
    elements into its memory."""
    import torch
    import tiled_matrix_multiply_amd as tmm
    i8 = t == "i8"
    G, M = len(sizes), sum(sizes)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def operand(count, rows, cols):
        flat = torch.full((count * rows * (cols + pad) + skew,), 127 if i8 else float("nan"), device="cuda",
                          dtype=dtype(t))
        view = flat[skew:].view(count, rows, cols + pad)
        if i8:
            view[:, :, :cols] = torch.randint(-128, 128, (count, rows, cols), device="cuda", generator=gen,
                                              dtype=torch.int8)
        else:
            view[:, :, :cols] = torch.randn(count, rows, cols, device="cuda", generator=gen).to(dtype(t))
        return flat[skew:], view[:, :, :cols]

    A, a = operand(1, M, K)
    B, b = operand(G, *((N, K) if nk else (K, N)))
    out = torch.randn(M * (N + pad) + skew, device="cuda", generator=gen).to(dtype(ct))
    C = out[skew:].view(M, N + pad)
    before = out.clone()
    cin = before[skew:].view(M, N + pad)[:, :N].double()
    bias_t = torch.randn(G, N, device="cuda", generator=gen) if bias else None
    sa = torch.rand(M, device="cuda", generator=gen) * 0.1 + 1e-3
    sb = torch.rand(G, N, device="cuda", generator=gen) * 1e-2 + 1e-3
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)).cuda()
    kw = dict(M=M, N=N, K=K, trans_b=nk, alpha=alpha, beta=beta, lda=K + pad, ldb=(K if nk else N) + pad, ldc=N + pad,
              epilogue=(tmm.GEMM_EPI_BIAS if bias else 0) | (tmm.GEMM_EPI_GELU if do_gelu else 0), bias=bias_t, kernel=kernel)
    print(f"[path] kernel {kernel} {t} {ct} {'NK' if nk else 'KN'} {sizes[:6]} {N} {K}", flush=True)
    if not i8:
        g.run_grouped(A, B, C, off, groups=G, a_type=t, **kw)
    elif grouped:
        g.run_grouped_i8(A, sa, B, sb, C, off, groups=G, c_type=ct, **kw)
    else:
        g.run_i8(A, sa, B, sb, C, c_type=ct, **kw)
    torch.cuda.synchronize()
    ref, D = torch.empty(M, N, device="cuda", dtype=torch.float64), torch.empty(M, N, device="cuda", dtype=torch.float64)
    r = 0
    for q, n in enumerate(sizes):
        rows = slice(r, r + n)
        r += n
        if n == 0:
            continue
        x, w = a[0, rows].double(), b[q].double()
        w = (w.t() if nk else w).contiguous()
        v = alpha * (x @ w)
        if i8:
            v = v * sa[rows, None].double() * sb[q].double()
            d = v.abs()
        else:
            d = alpha * (x.abs() @ w.abs())
        if beta:
            v, d = v + beta * cin[rows], d + (beta * cin[rows]).abs()
        if bias:
            v, d = v + bias_t[q].double(), d + bias_t[q].double().abs()
        ref[rows], D[rows] = (v * torch.special.ndtr(v) if do_gelu else v), d
    tol = (0 if i8 else K * 2.0 ** -23) + HALF_STEP[ct] + ((4 if i8 else 0) + (20 if do_gelu else 4)) * U32
    check(C[:, :N], ref, D, tol, ct, (kernel, t, nk, sizes[:6], N, K))
    same = out.clone()
    same[skew:].view(M, N + pad)[:, :N] = before[skew:].view(M, N + pad)[:, :N]
    assert torch.equal(same, before), "outside C"


# ------------------------------------------------------------------------- the mixed kernel --

def mixed(sizes, N, cus):
    """Large tiles kept whole, large tiles split, and small tiles in all."""
    large = sum((n + 127) >> 8 for n in sizes) * ceil(N, 256)
    small = sum(1 for n in sizes if 0 < n & 255 <= 128) * ceil(N, 128)
    rounds, rest = divmod(large, cus)
    over = small - (2 * (cus - rest) if rest else 0)
    whole = 10 * (rounds + (rest > 0)) + 4 * ceil(max(over, 0), cus)
    apart = 10 * rounds + 4 * ceil(small + 4 * rest, cus)
    split = rest if apart < whole else 0
    return large - split, split, 4 * split + small


ROWS = [1000, 0, 517, 1300, 260, 900]  # 16 rows of large tiles and three of small ones
MIXED = {
    "kept": (ROWS, 2568),
    "kept and split": (ROWS, 4104),
    "more pieces than workgroups": (ROWS + [100, 3, 128, 77, 0, 1, 64, 90, 11], 4104),
    "one group": ([4100], 4104),
}


@pytest.mark.parametrize("path", sorted(MIXED))
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16"), ("i8", "f32")])
def test_mixed(g, t, ct, nk, path):
    sizes, N = MIXED[path]
    cus = compute_units()
    kept, split, pieces = mixed(sizes, N, cus)
    if cus == 256:
        assert kept > 128 and (split > 0) == (path != "kept")
        assert (pieces > cus) == (path == "more pieces than workgroups")
    step = 16 if t == "i8" else 8
    N = ceil(N, step) * step
    for kernel in (AUTO, TILE_256):
        # 2 K tiles, the last one cut, and 8
        for K, do_gelu, beta in ((13 * step, False, -0.5), (57 * step, True, 0.0)):
            product(g, sizes, N, K, nk=nk, t=t, ct=ct, kernel=kernel, grouped=len(sizes) > 1, pad=step, do_gelu=do_gelu,
                    beta=beta, seed=K)


# -------------------------------------------------------------------- any alignment, K unsplit --

@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16"), ("i8", "f32")])
def test_any_alignment(g, t, ct, nk):
    """Odd sizes, leading dimensions and starts; widths and depths of less than one copied chunk."""
    for sizes, N, K in (([700, 1, 613], 1001, 75), ([700, 1, 613], 1001, 203), ([9000, 0, 10003], 5, 203),
                        ([9000, 0, 10003], 101, 5), ([1600, 900], 517, 1003)):
        rows = ceil(sum(sizes) + len(sizes) * 32, 64)
        assert rows * ceil(N, 64) > compute_units()
        for kernel in (AUTO, ANY):
            product(g, sizes, N, K, nk=nk, t=t, ct=ct, kernel=kernel, pad=3, skew=1, do_gelu=K == 75,
                    beta=0.5 if K == 203 else 0.0, seed=N + K)


# ------------------------------------------------------------------------------- streaming --

@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16"), ("i8", "f32")])
def test_streaming_64_rows(g, t, ct):
    """64 rows a workgroup: the columns of the last block moved back to the edge, and a last, partial
    step of K beside more blocks of K than waves."""
    for sizes, N, nk in (([64], 16385, False), ([50], 16386, False), ([1000], 1003, False), ([700, 0, 130, 64], 2003, False),
                         ([64], 8201, True)):
        rows, cus = 64, compute_units()
        tiles = ceil(sum(sizes), 64) if len(sizes) == 1 else ceil(sum(sizes) + len(sizes) * 32, 64)
        avg = ceil(sum(sizes), len(sizes))
        assert avg > (32 if len(sizes) == 1 else 24) and 4 * tiles * ceil(N, 32 if nk else 64) > 3 * cus
        for K in (203, 1003):
            K = 2 * K if t == "i8" else K
            product(g, sizes, N, K, nk=nk, t=t, ct=ct, kernel=STREAM, pad=1, skew=1, do_gelu=K < 500,
                    beta=0.5 if K < 500 else 0.0, seed=N + K)


# ------------------------------------------------------------------------------- gradients --

@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("t,ct", [("bf16", "bf16"), ("f16", "f32")])
def test_gradient_tiles_dealt_unevenly(g, t, ct, nk):
    """64 tiles or more a group, in a number that is no multiple of the XCDs'."""
    import torch
    for kernel, tile, N, K, sizes in ((ANY, 64, 837, 329, [70, 0, 33, 300, 1]), (TILE_64, 64, 840, 328, [70, 0, 33, 300, 1]),
                                      (TILE_128, 128, 1160, 840, [70, 0, 333]), (TILE_256, 256, 2120, 2056, [300, 70])):
        tiles = ceil(N, tile) * ceil(K, tile)
        assert tiles >= 64 and tiles % 8
        G, M = len(sizes), sum(sizes)
        gen = torch.Generator(device="cuda").manual_seed(N)
        A = torch.randn(M, K, device="cuda", generator=gen).to(dtype(t))
        D = torch.randn(M, N, device="cuda", generator=gen).to(dtype(t))
        C = torch.randn(G, *((N, K) if nk else (K, N)), device="cuda", generator=gen).to(dtype(ct))
        before, db = C.double(), torch.full((G, N), float("nan"), device="cuda")
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)).cuda()
        print(f"[path] gradient {kernel} {t} {ct} {N} {K}", flush=True)
        g.run_grouped_wgrad(A, D, C, off, groups=G, M=M, N=N, K=K, trans_b=nk, a_type=t, c_type=ct, alpha=0.5, beta=0.25,
                            dbias=db, kernel=kernel)
        torch.cuda.synchronize()
        r = 0
        for q, n in enumerate(sizes):
            a, d = A[r:r + n].double(), D[r:r + n].double()
            r += n
            x, y = (d, a) if nk else (a, d)
            v, den = 0.5 * (x.t().contiguous() @ y), 0.5 * (x.abs().t().contiguous() @ y.abs())
            v, den = v + 0.25 * before[q], den + 0.25 * before[q].abs()
            check(C[q], v, den, n * 2.0 ** -23 + HALF_STEP[ct] + 4 * U32, ct, (kernel, t, nk, q))
            check(db[q], d.sum(0), d.abs().sum(0), (n + 2) * U32, "f32", ("bias", kernel, q))
