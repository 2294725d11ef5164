"""Where the device cannot place a cluster of the decode's splits, the call goes through the workspace, which it asked
for, and is not refused."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from attn_fwd_02_gb300 import build
    out = str(tmp_path_factory.mktemp("cluster") / "launches")
    wraps = [f"-Xlinker=--wrap={f}" for f in (
        "cudaLaunchKernelExC", "cudaLaunchKernel", "__cudaLaunchKernel", "cudaGetLastError")]
    # code for the host alone runs here: the device's stays PTX
    r = subprocess.run([build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-O0", "-std=c++17",
                        "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", build.CSRC,
                        os.path.join(ROOT, "tests", "cluster_fallback.cu"), "-o", out, *wraps],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def launches(program, room, *sizes):
    r = subprocess.run([program, str(int(room)), *map(str, sizes)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    *lines, status = r.stdout.split("\n")[:-1]
    return lines, int(status.split()[1])


SIZES = [(1, 8, 8, 100), (2, 12, 12, 57), (8, 32, 8, 22)]  # B, H, Hkv, pages


@pytest.mark.parametrize("size", SIZES)
def test_clusters_where_they_fit(program, size):
    lines, status = launches(program, True, *size)
    assert status == 0 and len(lines) == 1
    kind, grid, *rest = lines[0].split()
    n = int(grid.split(",")[0])
    assert kind == "cluster" and 1 < n <= 16 and rest == ["splits", str(n), "chunk", "0", "cluster", "1"]


@pytest.mark.parametrize("size", SIZES)
def test_the_workspace_where_they_do_not(program, size):
    B, H, Hkv, pages = size
    lines, status = launches(program, False, *size)
    assert status == 0
    (a, b) = (line.split() for line in lines)
    chunk = int(a[5])
    splits = -(-pages // chunk)
    assert a == ["plain", f"{splits},{Hkv},{B}", "splits", str(splits), "chunk", str(chunk), "cluster", "0"]
    assert b == ["dependent", f"{-(-B * H // 4)},1,1", "splits", str(splits), "chunk", str(chunk), "cluster", "0"]
