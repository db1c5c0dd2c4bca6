"""The count of clusters that fit on a device, over a CUDA runtime made of answers: built and
run on the CPU."""
import os
import shutil
import subprocess

import pytest

from sparse_attention_fp4_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_sizes_that_cannot_be_placed(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    nvcc = build._nvcc()
    objs = []
    # (a .cpp file goes to the host compiler, with CUDA's headers)
    for src in (os.path.join(build.CSRC, "host_util.cu"), os.path.join(HERE, "host", "cluster_sizes.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([nvcc, "-c", src, "-o", objs[-1], "-O3", "-std=c++17", "-I", os.path.join(build.ROOT, "include")] + build.ARCH,
                       check=True)
    exe = str(tmp_path / "cluster_sizes")
    subprocess.run([cxx, "-o", exe] + objs + ["-lpthread"], check=True)
    got = subprocess.run([exe], capture_output=True, text=True)
    assert got.returncode == 0 and got.stdout.strip() == "OK", got.stdout
