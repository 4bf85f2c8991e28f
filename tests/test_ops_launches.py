"""Host tests of what the feed-forward operators launch: cp_ops.cpp is compiled
with launchers that print what they are asked for (tests/sim/cp_ops_launches.cpp)."""
import os
import random
import re
import shutil
import subprocess
import time

import pytest

from ops_kernels import CASES

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


# -------------------------------------------------- outputs that overlap inputs

@pytest.fixture(scope="module")
def many(launches):
    """The same program, many lines at a time: [(status, error text)]."""
    exe = launches.__closure__[0].cell_contents

    def call(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True, timeout=60).stdout
        found = [re.search(r"status=(-?\d+) ?(.*)$", line) for line in out.splitlines()]
        assert len(found) == len(lines) and all(found)
        return [(int(m.group(1)), m.group(2)) for m in found]
    return call


def taken(p, rows, cols, ld, es=2, count=1, stride=0):
    """The bytes of a matrix (or of `count` of them)."""
    return {p + (e * stride + r * ld) * es + i for e in range(count) for r in range(rows) for i in range(cols * es)} if p else set()


def test_overlap_against_bytes(many):
    """Y and pre at random places in a small buffer: refused if and only if they share a byte with an input or
    each other; Y may be R itself."""
    rng = random.Random(5)
    lines, want = [], []
    for _ in range(4000):
        M, K, N, E = rng.randint(1, 5), rng.randint(1, 6), rng.randint(1, 6), rng.choice([0, 0, 1, 3])
        base, far = 1 << 20, 1 << 30

        def at(share):
            return base + 2 * rng.randint(0, 80) if rng.random() < share else far + (rng.randint(1, 1 << 10) << 16)
        X, W, R, Y, P, b = at(0.5), at(0.3), at(0.3), base + 2 * rng.randint(0, 80), at(0.3), at(0.2)
        off = far - (1 << 24) if rng.random() < 0.9 else base + 4 * rng.randint(0, 40)
        R, P, b = (0 if rng.random() < 0.5 else v for v in (R, P, b))
        lx, lw, lr, ly, lp = K + rng.randint(0, 9), N + rng.randint(0, 3), N + rng.randint(0, 9), N + rng.randint(0, 9), N + rng.randint(0, 9)
        if rng.random() < 0.5:  # views of one buffer
            ld = max(K, N) + rng.randint(0, 12)
            lx, lr, ly, lp = ld, ld, ld, ld
        if E:
            R = 0
        if R and rng.random() < 0.3:
            Y, ly = R, lr
        sw = (K - 1) * lw + N + rng.randint(0, 4)
        lines.append(f"linear 1 {M} {K} {N} {E} 0 {X} {lx} {W} {lw} {sw} {b} {off} {R} {lr} {Y} {ly} {P} {lp}")
        ins = {"X": taken(X, M, K, lx), "W": taken(W, K, N, lw, count=max(E, 1), stride=sw), "bias": taken(b, 1, N * max(E, 1), 0),
               "offsets": taken(off, 1, E + 1, 0, es=4) if E else set(), "R": taken(R, M, N, lr)}
        y, pre = taken(Y, M, N, ly), taken(P, M, N, lp)
        bad = bool(y & pre) or any(bool(pre & v) for v in ins.values())
        bad = bad or any(bool(y & v) for k, v in ins.items() if not (k == "R" and Y == R and (ly == lr or M == 1)))
        want.append(bad)
    got = many(lines)
    assert 0.1 < sum(want) / len(want) < 0.9
    for line, bad, (status, text) in zip(lines, want, got):
        assert (status == -1 and "overlaps" in text) if bad else status == 0, (line, bad, status, text)


def test_norm_overlap_against_bytes(many):
    rng = random.Random(6)
    lines, want = [], []
    for _ in range(2000):
        M, N = rng.randint(1, 5), rng.randint(1, 6)
        X, Y, w, b = (1 << 20) + 2 * rng.randint(0, 60), (1 << 20) + 2 * rng.randint(0, 60), *(
            rng.choice([0, 1 << 24, (1 << 20) + 2 * rng.randint(0, 60)]) for _ in range(2))
        lx = N + rng.randint(0, 9)
        ly = lx if rng.random() < 0.6 else N + rng.randint(0, 9)
        if rng.random() < 0.3:
            Y = X
        lines.append(f"norm 1 {M} {N} {X} {lx} {w} {b} {Y} {ly}")
        y = taken(Y, M, N, ly)
        bad = bool(y & (taken(w, 1, N, 0) | taken(b, 1, N, 0)))
        want.append(bad or (bool(y & taken(X, M, N, lx)) and not (Y == X and (ly == lx or M == 1))))
    for line, bad, (status, text) in zip(lines, want, many(lines)):
        assert (status == -1 and "overlaps" in text) if bad else status == 0, (line, bad, status, text)
    assert 0.1 < sum(want) / len(want) < 0.9


def test_overlap_of_large_views(many):
    """Interleaved views of 2^30 rows, whose patterns differ or repeat late, are decided at once."""
    M, far = 1 << 30, 1 << 58
    t0 = time.time()
    got = many([
        f"linear 1 {M} 8 8 0 0 {1 << 20} 16 {far} 8 0 0 0 0 0 {(1 << 20) + 16} 16 0 0",           # columns 8 .. 15 of the same rows
        f"linear 1 {M} 8 8 0 0 {1 << 20} 16 {far} 8 0 0 0 0 0 {(1 << 20) + 14} 16 0 0",           # 7 .. 14
        # strides 32 bytes apart: rows of 16 bytes, 16 - 32 q bytes from each other, never meet; 24 - 32 q do
        f"linear 1 {M} 8 8 0 0 {1 << 20} 4194304 {far} 8 0 0 0 0 0 {(1 << 20) + 16} 4194288 0 0",
        f"linear 1 {M} 8 8 0 0 {1 << 20} 4194304 {far} 8 0 0 0 0 0 {(1 << 20) + 24} 4194288 0 0",
        # 2 bytes apart: they meet after seven rows, or only after 4194304 - 7
        f"linear 1 {M} 8 8 0 0 {1 << 20} 4194304 {far} 8 0 0 0 0 0 {(1 << 20) + 16} 4194303 0 0",
        f"linear 1 {M} 8 8 0 0 {1 << 20} 4194303 {far} 8 0 0 0 0 0 {(1 << 20) + 16} 4194304 0 0",
    ])
    assert [s for s, _ in got] == [0, -1, 0, -1, -1, -1] and time.time() - t0 < 20


# -------------------------------------------------- the kernels the choice picks

def launches_of(out):
    out = re.sub(r":(threads|n[xwd])=\d+|:direct=1\b|:split=1\b", "", " ".join(out))
    return out.replace(":layout=0", ":NN").replace(":layout=1", ":NT").replace(":layout=2", ":TN")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:10])))
def test_choice(launches, case):
    out, status = launches(*case[:10])
    assert status == CP_OK and launches_of(out) == case[10]


def test_every_kernel_is_launched():
    """Each configuration, dense and by expert, in both types and weight layouts, alone and for both gradients at once;
    those of a product alone also split."""
    got = set()
    for c in CASES:
        for w, layout, split in re.findall(r"((?:product|gradients):\w+)(?::([NT]{2}))?(:split=\d+)?", c[10]):
            got.add((c[1], c[5] > 0, w, layout or c[6], bool(split)))
        if "gemv" in c[10]:
            got.add((c[0], c[1], "gemv", c[6]))
    tiles = {BF16: ("256x256", "128x256", "128x128", "64x128", "64x64"), F32: ("128x128", "64x128", "64x64")}
    want = {(d, g, f"gradients:{t}", wt, False) for d in tiles for g in (False, True) for t in tiles[d] for wt in (0, 1)}
    want |= {(d, g, f"product:{t}", layout, split) for d in tiles for g in (False, True) for t in tiles[d]
             for layout in ("NN", "NT", "TN") for split in (False, True)}
    want |= {(d, g, "product:16x128", layout, split) for d in tiles for g in (False, True) for layout in ("NN", "NT")
             for split in (False, True)}
    want |= {("forward", d, "gemv", wt) for d in tiles for wt in (0, 1)}
    assert want <= got, sorted(want - got, key=str)
