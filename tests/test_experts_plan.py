"""The host side of the calls of gemm_experts.h without a GPU: xapi.cpp under the address and
undefined-behaviour sanitizers, with launchers that print what they are asked to launch
(tests/asan/experts_driver.cpp), at sizes whose products pass 32 and 64 bits."""
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
    """plan(call, ...): the words of each call's answer."""
    script = os.path.join(ROOT, "tests", "asan", "experts.sh")
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
        out = [[int(w) if w.lstrip("-").isdigit() else w for w in line.split()] for line in r.stdout.splitlines()]
        assert len(out) == len(calls)
        return out

    return run


def words(*args):
    return " ".join(str(a) for a in args)


def mx(M, N, K, *, groups=1, kernel=0, lda=-1, ldb=-1, ldc=-1, ldsa=-1, ldsb=-1, stride=-1, skew=0, ct=BF16, epi=0):
    return words("mx", kernel, groups, M, N, K, lda, ldb, ldc, ldsa, ldsb, stride, skew, ct, epi)


def stream(rows, columns):
    return [OK, "stream", rows, columns]


def tile(n):
    return [OK, "tile", n]


# what AUTO takes on both sides of each border of its rule, with 256 compute units; tiles: 1 64 x 64 (4 with
# a third stage), 2 128 x 128, 3 256 x 256 mixed with 128 x 128
@pytest.mark.parametrize("args,launch", [
    # one token up to eight stream whatever the width, in half as many columns
    ((1, 65536, 2048, {}), stream(16, 16)), ((8, 65536, 2048, {}), stream(16, 16)), ((9, 65536, 2048, {}), tile(1)),
    # more rows of one group: three rounds of 16 x 16, two of 16 x 32, one of 32 x 32
    ((9, 4096, 4096, {}), stream(16, 16)), ((9, 4112, 4096, {}), stream(16, 32)), ((16, 8192, 4096, {}), stream(16, 32)),
    ((16, 8224, 4096, {}), stream(16, 16)), ((16, 12288, 4096, {}), stream(16, 16)), ((16, 12304, 4096, {}), stream(16, 32)),
    ((16, 16384, 4096, {}), stream(16, 32)), ((16, 16416, 4096, {}), tile(4)),
    ((128, 2048, 4096, {}), stream(32, 32)), ((128, 2080, 4096, {}), tile(4)),
    ((256, 1024, 4096, {}), stream(32, 32)), ((257, 1024, 4096, {}), tile(4)), ((48, 8192, 4096, {}), tile(4)),
    # the rows and columns of a streaming workgroup that the tiles cannot take
    ((48, 8192, 4096, dict(skew=1)), stream(64, 32)), ((32, 8192, 4096, dict(skew=1)), stream(32, 32)),
    ((37, 4104, 4128, dict(skew=1)), stream(16, 32)),
    # many groups: 2.5 tiles a compute unit with up to 4 rows to a group, 1.25 with more, a quarter with up to 128
    ((128, 2240, 2048, dict(groups=32)), stream(16, 32)), ((128, 2304, 2048, dict(groups=32)), tile(1)),
    ((160, 1024, 2048, dict(groups=32)), stream(16, 32)), ((160, 1088, 2048, dict(groups=32)), tile(1)),
    ((512, 256, 2048, dict(groups=8)), stream(16, 32)), ((512, 448, 2048, dict(groups=8)), tile(1)),
    ((16, 1024, 2048, dict(groups=4)), stream(16, 16)),
    # large tiles from 5/8 of a round, with groups from 3/8 and 160 rows to a group
    ((2560, 4096, 1024, {}), tile(3)), ((2559, 4096, 1024, {}), tile(2)),
    ((1280, 5120, 1024, dict(groups=8)), tile(3)), ((1272, 5120, 1024, dict(groups=8)), tile(2)),
    ((1280, 4864, 1024, dict(groups=8)), tile(2)),
    # 128 x 128 from 13/16 of a round, with GELU from 9/8, and from 96 rows to a group
    ((1024, 3328, 2048, {}), tile(2)), ((1024, 3200, 2048, {}), tile(1)),
    ((1024, 4608, 2048, dict(epi=2)), tile(2)), ((1024, 4480, 2048, dict(epi=2)), tile(1)),
    ((1536, 2048, 2048, dict(groups=16)), tile(2)), ((1520, 2048, 2048, dict(groups=16)), tile(1)),
    ((96, 28672, 2048, {}), tile(2)), ((95, 28672, 2048, {}), tile(1)),
    # a third stage for a long K and up to two tiles a compute unit
    ((1024, 2048, 4096, {}), tile(4)), ((1024, 2112, 4096, {}), tile(1)), ((1024, 2048, 4064, {}), tile(1)),
])
def test_auto(plan, args, launch):
    M, N, K, kw = args
    assert plan(mx(M, N, K, **kw))[0] == launch


def test_what_the_tiles_cannot_take_is_streamed(plan):
    """Alignment, and scales past 2^32 bytes."""
    for kw in (dict(skew=1), dict(ldc=4099), dict(lda=2080 + 2), dict(ldsa=65), dict(ldsb=70), dict(stride=4096 * 2048 + 2)):
        got = plan(mx(4096, 4096, 2048, groups=2, **kw), mx(4096, 4096, 2048, groups=2, kernel=tmm.GEMM_GROUPED_MFMA_256, **kw))
        assert got[0][:2] == [OK, "stream"] and got[1] == [U], kw
    got = plan(mx(2 ** 22, 64, 32, ldsa=1024 - 16), mx(2 ** 22, 64, 32, ldsa=1024), mx(2 ** 22, 64, 32, ldsa=2 ** 23 + 16))
    assert got[0][1] == "tile" and got[1][1] == "stream" and got[2] == [U]


def test_long_rows(plan):
    """Rows of up to 2^23 bytes; one row alone may have any leading dimension."""
    most = 2 ** 24
    assert [a[0] for a in plan(mx(2, 64, 64, lda=most), mx(2, 64, 64, lda=most + 32), mx(64, 2, 64, ldb=most + 32))] == [OK, U, U]
    for lda in (most + 32, 2 ** 40, 2 ** 62, 2 ** 63 - 32):
        got = plan(mx(1, 64, 64, lda=lda), mx(1, 64, 64, lda=lda, kernel=tmm.GEMM_GROUPED_MFMA_64))
        assert got == [stream(16, 16), [U]], lda


def test_what_cannot_be_counted(plan):
    got = plan(mx(MOST, MOST, 32, groups=65535, stride=0), mx(MOST, MOST, 32), mx(2 ** 22, 2 ** 19, 32),
               mx(2 ** 22, 2 ** 20, 32), mx(MOST, 16, MOST // 32 * 32, stride=0), mx(MOST + 1, 16, 32),
               mx(2 ** 26, 2 ** 14, 32, kernel=tmm.GEMM_GROUPED_STREAM))
    assert [a[0] for a in got] == [U, U, OK, U, U, U, OK]


def test_moves_of_any_size(plan):
    """Pairs are counted in 31 bits; addresses in 64."""
    every = [OK] * 4 + ["dispatch", "combine", "grad", "quantize"]
    got = plan(words("moves", MOST, 1, 32, 32, MOST, BF16), words("moves", MOST // 32, 32, 64, 64, MOST, F32),
               words("moves", MOST, 2, 32, 32, MOST, BF16), words("moves", 1, MOST, 32, 32, 5, F16),
               words("moves", 2, MOST, 32, 32, 5, F16), words("moves", 4, 2, MOST // 32 * 32, MOST, 8, BF16),
               words("moves", 4, 2, 64, 2 ** 40, 8, BF16))
    assert got[0] == every and got[1] == every and got[2] == [U] * 4 and got[3] == every and got[4] == [U] * 4
    assert got[5] == every and got[6] == every


def test_router_of_any_size(plan):
    got = plan(words("route", 2 ** 29, 1024, 3, 1, 1, 1024, BF16, 0, 1), words("route", 2 ** 29 + 1, 8, 1, 1, 1, 8, F32, 0, 0),
               words("route", 2 ** 29, 8, 4, 1, 1, 8, F32, 0, 0), words("route", 0, 8, 4, 8, 4, 8, F32, 1, 0),
               words("route", 64, 8, 4, 8, 4, 8, F32, 1, 0), words("route", 65, 8, 4, 8, 4, 8, F32, 1, 0),
               words("route", 10, 1024, 32, 64, 2, 1024, F16, 1, 1), words("route", 10, 1024, 32, 128, 2, 1024, F16, 1, 1),
               words("route", 10, 1024, 16, 128, 2, 1024, F16, 1, 1))
    assert got[0] == [2 ** 33, OK, OK, "route", "grad"]
    assert got[1] == [U, U, U] and got[2][1:] == [U, U]
    assert got[3] == [0, OK, OK, "route"]  # no gradient without tokens
    assert got[4] == [0, OK, OK, "route", "grad"] and got[5] == [5 * 16, OK, OK, "route", "grad"]
    assert got[6] == [0, OK, OK, "route", "grad"] and got[7] == [0, V, OK, "grad"]  # 16 are left
    assert got[8] == [0, U, OK, "grad"]
