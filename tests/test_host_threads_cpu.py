"""Several host threads on one stream, and on several, without a GPU (host_threads.cpp)."""

import os
import subprocess

import pytest

from newton_schulz_07_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host_threads(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("host") / "host_threads")
    rocm = os.path.dirname(os.path.dirname(build.hipcc()))
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-pthread", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(rocm, "include"), "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC,
                    os.path.join(HERE, "host_threads.cpp"),
                    *(os.path.join(build.CSRC, f) for f in ("ns_host.cpp", "ns_api.cpp", "ns_sublayer.cpp")),
                    "-o", exe], check=True, timeout=300)
    return exe


def test_calls_of_several_threads_keep_their_launches_together(host_threads):
    r = subprocess.run([host_threads], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
