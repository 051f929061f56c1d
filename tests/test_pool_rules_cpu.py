"""The rule by which the pool's gradients take one kernel or the other, as the launcher
computes it: the GPU tests' sizes reach the kernel that they are for."""

import os
import shutil
import subprocess

import pytest

from test_gpu_pool_grads import LONG, SPLIT

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                    reason="nvcc not available")
def test_sizes_reach_the_kernels_they_test(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = tmp_path / "pool_rules_check"
    src = os.path.join(ROOT, "tests", "host", "pool_rules_check.cu")
    b = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                        os.path.join(ROOT, "include"), "-o", str(exe), src], capture_output=True, text=True, timeout=600)
    assert b.returncode == 0, b.stderr[-3000:]
    sizes = [c[:5] for c in SPLIT + LONG] + [(2048, 11008, 4096, 64, 4), (1003, 1000, 576, 24, 6)]
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, s)) for s in sizes), capture_output=True, text=True, timeout=120)
    want = ["split"] * len(SPLIT) + ["split" if c[5] else "whole" for c in LONG] + ["whole", "whole"]
    assert r.stdout.split() == want
