"""The host side of the grouped and 8-bit integer calls without a GPU: gapi.cpp under the address and
undefined-behaviour sanitizers, with launchers that print what they are asked to launch
(tests/asan/grouped_driver.cpp), and the size checks that the library exports."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
tmm = pytest.importorskip("tiled_matrix_multiply_amd")

F16, BF16, F32 = tmm.GEMM_F16, tmm.GEMM_BF16, tmm.GEMM_F32
OK, V, U = tmm.GEMM_OK, tmm.GEMM_ERR_INVALID_VALUE, tmm.GEMM_ERR_UNSUPPORTED
MOST = 2 ** 31 - 1024  # the largest dimension


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(call, ...): the (status, launch) of each call; a launch is ("tile", number), ("stream",
    rows, waves) or None."""
    script = os.path.join(ROOT, "tests", "asan", "grouped.sh")
    if shutil.which("bash") is None or not os.path.exists("/opt/rocm/llvm/bin/clang"):
        pytest.skip("no ROCm clang")
    if not os.path.exists(script):
        pytest.skip("tests/asan is not in this copy of the tree")
    exe = str(tmp_path_factory.mktemp("plan") / "driver")
    r = subprocess.run(["bash", script, exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]

    def run(*calls):
        r = subprocess.run([exe], input="\n".join(calls), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and "runtime error" not in r.stderr, r.stderr[-4000:]
        out = []
        for line in r.stdout.splitlines():
            w = line.split()
            launch = {"none": None, "tile": ("tile", int(w[2])) if w[1] == "tile" else None,
                      "stream": ("stream", int(w[2]), int(w[3])) if w[1] == "stream" else None}[w[1]]
            out.append((int(w[0]), launch))
        assert len(out) == len(calls)
        return out

    return run


def call(op, M, N, K, *, groups=1, kernel=0, nk=True, lda=-1, ldb=-1, ldc=-1, stride=-1, skew=0, t=BF16,
         ct=BF16, dbias=False):
    return " ".join(str(int(v)) if not isinstance(v, str) else v for v in
                    (op, kernel, groups, M, N, K, nk, lda, ldb, ldc, stride, skew, t, ct, dbias))


# ------------------------------------------------------------------- sizes that cannot be counted --

def far(i):
    return i << 60


def test_checks_refuse_what_the_calls_refuse():
    """Tiles past 31 bits: the argument checks answer as the calls do."""
    def products(M, N, groups, i8=0):
        return tmm.gemm_check_args_grouped(groups, far(1), M, N, 8, 1, far(2), 8, far(5), far(3), 8, 0, far(6),
                                           far(4), N, i8, BF16, BF16, 0, None)

    def gradient(N, K, groups, dbias=None):
        return tmm.gemm_check_args_grouped_wgrad(groups, far(1), 40, N, K, 0, far(2), K, far(3), N, far(4), N,
                                                 N * K, BF16, BF16, dbias)

    for i8 in (0, 1):
        assert products(2 ** 21, 2 ** 21, 1, i8) == OK
        assert products(MOST, MOST, 1, i8) == U and products(MOST, MOST, 65535, i8) == U
        assert products(2 ** 22, 2 ** 20, 1, i8) == OK and products(2 ** 22, 2 ** 21, 1, i8) == U
        assert products(4096, 2 ** 25, 4096, i8) == U and products(4096, 2 ** 24, 4096, i8) == OK
    # 2^15 groups of 2^8 x 2^8 tiles are 2^31; a last round of 8 for each row of tiles of a group
    assert gradient(2 ** 14, 2 ** 14, 2 ** 14) == OK and gradient(2 ** 14, 2 ** 14, 2 ** 15) == U
    assert gradient(MOST, MOST, 1) == U
    # the product of the tiles and the groups passes 64 bits
    for groups in (8192, 2 ** 14, 65535):
        assert gradient(2 ** 30, 2 ** 30, groups) == U, groups


def test_calls_refuse_them(plan):
    got = plan(call("wgrad", 40, MOST, MOST, groups=65535, nk=False), call("wgrad", 40, MOST, MOST, groups=65535),
               call("wgrad", 40, 2 ** 30, 2 ** 30, groups=2 ** 14, nk=False),
               call("grouped", MOST, MOST, 8, groups=65535, stride=0), call("i8", MOST, MOST, 16))
    assert got == [(U, None)] * 5
    # too many of the streaming kernel's workgroups, but not of the tiles
    got = plan(call("grouped", 4096, 2 ** 24 + 8, 96, groups=4096, stride=0),
               call("grouped", 4096, 2 ** 24 + 8, 96, groups=4096, stride=0, kernel=tmm.GEMM_GROUPED_STREAM),
               call("grouped", 4096, 2 ** 23, 96, groups=4096, stride=0))
    assert got[0] == (OK, ("tile", 0)) and got[1] == (U, None) and got[2][1][0] == "stream"


# -------------------------------------------------------------------------- leading dimensions --

def test_rows_too_long_for_lane_offsets(plan):
    """Rows past 2^23 bytes go to the kernel with 64-bit offsets, up to the leading dimensions whose
    bytes pass 63 bits (which one row alone may have)."""
    most = 2 ** 23 // 2
    for lda, launch in ((most, "stream"), (most + 8, "tile"), (2 ** 40, "tile"), (2 ** 62, "tile"), (2 ** 62 + 8, "tile"),
                        (2 ** 63 - 8, "tile")):
        st, got = plan(call("grouped", 1, 64, 256, lda=lda))[0]
        assert st == OK and got[0] == launch, lda
        if launch == "tile":
            assert got[1] in (0, 5), lda  # any alignment and length
    for kernel in (tmm.GEMM_GROUPED_MFMA_64, tmm.GEMM_GROUPED_MFMA_256, tmm.GEMM_GROUPED_STREAM):
        got = plan(call("grouped", 1, 64, 64, lda=most, kernel=kernel), call("grouped", 1, 64, 64, lda=2 ** 62, kernel=kernel),
                   call("grouped", 64, 1, 1, nk=False, ldb=2 ** 62, kernel=kernel))
        assert [st for st, _ in got] == [OK, U, U], kernel
    got = plan(call("i8", 1, 64, 64, lda=2 ** 23), call("i8", 1, 64, 64, lda=2 ** 23 + 16))
    assert got[0][1][0] == "stream" and got[1][1] == ("tile", 5)


# ---------------------------------------------------------------------------- the kernel choice --

def tile(n):
    return ("tile", n)


# what AUTO takes on both sides of each border of its rule, with 256 compute units; tiles: 0 any alignment
# (5 with K split), 1 64 x 64 (4 with more stages), 2 128 x 128, 3 256 x 256
@pytest.mark.parametrize("args,launch", [
    # few rows a group: 8 and 4 where 128 x 128 tiles would fill the compute units ...
    (("grouped", 256, 2048, 2048, dict(groups=32)), "stream"), (("grouped", 288, 2048, 2048, dict(groups=32)), tile(3)),
    (("grouped", 128, 2048, 2048, dict(groups=32, nk=False)), "stream"),
    (("grouped", 160, 2048, 2048, dict(groups=32, nk=False)), tile(3)),
    # ... 32 and 64 where not, 24 or 48 (64) without tiles for the alignment
    (("grouped", 32, 8192, 4096, dict()), "stream"), (("grouped", 33, 8192, 4096, dict()), tile(4)),
    (("grouped", 64, 8192, 4096, dict(nk=False)), "stream"), (("grouped", 65, 8192, 4096, dict(nk=False)), tile(4)),
    (("grouped", 48, 8192, 4096, dict(skew=2)), "stream"), (("grouped", 49, 8192, 4096, dict(skew=2)), tile(5)),
    (("grouped", 768, 2048, 2048, dict(groups=32, skew=2)), "stream"),
    (("grouped", 800, 2048, 2048, dict(groups=32, skew=2)), tile(0)),
    # at most a quarter of the compute units in 64 x 64 tiles
    (("grouped", 512, 512, 1824, dict()), "stream"), (("grouped", 512, 576, 1824, dict()), tile(4)),
    # a K of one and a half K tiles
    (("grouped", 8192, 8192, 96, dict()), tile(0)), (("grouped", 8192, 8192, 104, dict()), tile(3)),
    (("i8", 8192, 8192, 192, dict()), tile(0)), (("i8", 8192, 8192, 208, dict()), tile(3)),
    # half a round of 256 x 256 tiles, 9/16 of one of 128 x 128
    (("grouped", 2048, 4096, 2048, dict()), tile(3)), (("grouped", 2048, 3840, 2048, dict()), tile(2)),
    (("grouped", 1536, 1536, 2048, dict()), tile(2)), (("grouped", 1536, 1408, 2048, dict()), tile(1)),
    # 64 x 64: more stages up to one tile a compute unit
    (("grouped", 1024, 1024, 2048, dict()), tile(4)), (("grouped", 1024, 1088, 2048, dict()), tile(1)),
    # gradients: large tiles from 5/8 of a round, 128 x 128 from half of one
    (("wgrad", 4096, 2560, 4096, dict()), tile(3)), (("wgrad", 4096, 2304, 4096, dict()), tile(2)),
    (("wgrad", 4096, 1024, 2048, dict()), tile(2)), (("wgrad", 4096, 1024, 1920, dict()), tile(1)),
    (("wgrad", 4096, 1024, 1024, dict()), tile(4)), (("wgrad", 4096, 1024, 1088, dict()), tile(1)),
    # ... narrow ones of few rows, and those without tiles for the alignment
    (("wgrad", 256, 2048, 184, dict()), tile(5)), (("wgrad", 257, 2048, 184, dict()), tile(4)),
    (("wgrad", 256, 2048, 192, dict()), tile(4)), (("wgrad", 4096, 2560, 4096, dict(skew=2)), tile(0)),
    # the sizes of test_gpu_grouped_paths.py
    (("grouped", 3977, 2568, 104, dict(groups=6)), tile(3)), (("grouped_i8", 4451, 4112, 208, dict(groups=15)), tile(3)),
    (("i8", 4100, 4112, 208, dict()), tile(3)), (("grouped", 1314, 1001, 75, dict(groups=3, lda=78, skew=2)), tile(0)),
    (("grouped", 19003, 5, 203, dict(groups=3, lda=206, skew=2)), tile(0)),
    (("grouped", 64, 16385, 203, dict(nk=False, skew=2)), ("stream", 64)),
    (("grouped", 1000, 1003, 203, dict(nk=False, skew=2, kernel=5)), ("stream", 64)),
])
def test_auto(plan, args, launch):
    op, M, N, K, kw = args
    st, got = plan(call(op, M, N, K, **kw))[0]
    assert st == OK
    assert got[0] == launch if isinstance(launch, str) else got[:len(launch)] == launch
