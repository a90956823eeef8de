"""Grids of the layer operators' launches at the largest sizes gc.h accepts, without a GPU:
tests/abi_c/launch_sizes.cpp stands in for hipLaunchKernel and checks what the library asks for."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "collective_communication_reduction_amd")


def test_no_launch_holds_more_than_32_bits_of_work_items(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = str(tmp_path / "launch_sizes")
    p = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
                        "-isystem", os.path.join(rocm, "include"), os.path.join(ROOT, "tests", "abi_c", "launch_sizes.cpp"), "-o", exe,
                        f"-L{PKG}", "-lgc", f"-L{os.path.join(rocm, 'lib')}", "-lamdhip64", f"-Wl,-rpath,{PKG}",
                        f"-Wl,-rpath,{os.path.join(rocm, 'lib')}"], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "0 failures" in p.stdout, (p.stdout[-3000:], p.stderr[-2000:])
