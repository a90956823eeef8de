"""Which elements of a row each piece of its 16-byte units writes where sums are added to it, without a GPU:
tests/abi_c/unit_pieces.cpp counts them with the kernels' own index rules."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_element_is_written_once(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = str(tmp_path / "unit_pieces")
    p = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
                        f"-I{os.path.join(ROOT, 'collective_communication_reduction_amd', 'csrc')}", "-isystem", os.path.join(rocm, "include"),
                        os.path.join(ROOT, "tests", "abi_c", "unit_pieces.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-3000:]
    p = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and "0 failures" in p.stdout, p.stdout[-3000:]
