"""Host tests of what the feed-forward operators launch: cp_ops.cpp is compiled
with launchers that print what they are asked for (tests/sim/cp_ops_launches.cpp)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "sim", "cp_ops_launches.cpp")
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
BF16, F32 = 1, 0
CP_OK, CP_ERR_SHAPE = 0, -2


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """f(op, dtype, M, K, N, E, w_trans, act, parts, aligned) -> (launches, status)."""
    hipcc = HIPCC if os.path.exists(HIPCC) else shutil.which("hipcc")
    if not hipcc:
        pytest.skip("no hipcc")
    exe = str(tmp_path_factory.mktemp("launches") / "launches")
    subprocess.run([hipcc, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    SRC, "-o", exe], check=True, timeout=300)

    def call(op, dtype, M, K, N, E=0, wt=0, act=0, parts=7, aligned=1):
        line = f"{op} {dtype} {M} {K} {N} {E} {wt} {act} {parts} {aligned}\n"
        out = subprocess.run([exe], input=line, capture_output=True, text=True, check=True, timeout=60).stdout.split()
        assert out[-1].startswith("status="), (line, out)
        return out[:-1], int(out[-1][7:])
    return call


# The grid of a launch is counted in threads, in 32 bits, and wraps around without
# an error: each of these has to stay below, by larger tiles, or to be refused.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("op, M, K, N, E", [
    ("forward", 1 << 30, 8, 8, 0), ("forward", 1 << 30, 8, 64, 0), ("forward", 1 << 29, 8, 72, 0),
    ("forward", 1 << 22, 64, 1 << 22, 0), ("forward", 1 << 30, 8, 1 << 22, 0), ("forward", 4096, 8, 1 << 20, 4096),
    ("forward", 1 << 30, 8, 72, 7), ("forward", 1 << 28, 512, 4096, 4096), ("backward", 1 << 30, 8, 8, 0),
    ("backward", 1 << 30, 64, 64, 5), ("backward", 1 << 30, 8, 128, 0), ("backward", 1 << 16, 1 << 12, 1 << 14, 4096),
    ("backward", 1 << 16, 1 << 18, 1 << 14, 4096), ("backward", 4096, 8, 1 << 22, 4096)])
@pytest.mark.parametrize("wt", [0, 1])
def test_products_fit_a_grid(launches, op, M, K, N, E, dtype, wt):
    out, status = launches(op, dtype, M, K, N, E, wt=wt)
    threads = [int(t) for t in re.findall(r"threads=(\d+)", " ".join(out))]
    assert all(0 < t < 1 << 32 for t in threads), out
    assert status in (CP_OK, CP_ERR_SHAPE)
    if E == 0 and M * N <= 1 << 37:  # (what memory holds)
        assert status == CP_OK and threads, out
