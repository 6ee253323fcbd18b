"""How a stream's workspace grows, without a GPU (host_workspace.cpp)."""

import os
import subprocess

from newton_schulz_07_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_workspace_that_grows_slowly_holds_little(tmp_path):
    exe = str(tmp_path / "host_workspace")
    rocm = os.path.dirname(os.path.dirname(build.hipcc()))
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-pthread", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(rocm, "include"), "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC,
                    os.path.join(HERE, "host_workspace.cpp"), os.path.join(build.CSRC, "ns_host.cpp"), "-o", exe],
                   check=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
