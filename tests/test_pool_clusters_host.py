"""The clusters that a fork and a compaction launch, over a CUDA runtime made of answers: run on the CPU."""
import os
import shutil
import subprocess

import pytest

from sparse_attention_fp4_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_devices_with_and_without_clusters_of_sixteen(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    build.build()
    objs = [os.path.join(build.BUILD, name + ".o") for name in ("api_beam", "beam_select", "copy_pages", "page_pool", "host_util")]
    objs.append(str(tmp_path / "pool_clusters.o"))
    # (a .cpp file goes to the host compiler, with CUDA's headers)
    subprocess.run([build._nvcc(), "-c", os.path.join(HERE, "host", "pool_clusters.cpp"), "-o", objs[-1], "-O1", "-std=c++17", "-I",
                    os.path.join(build.ROOT, "include")], check=True)
    exe = str(tmp_path / "pool_clusters")
    subprocess.run([cxx, "-o", exe] + objs + ["-lpthread"], check=True)
    got = subprocess.run([exe], capture_output=True, text=True)
    assert got.returncode == 0 and got.stdout.strip() == "OK", got.stdout
