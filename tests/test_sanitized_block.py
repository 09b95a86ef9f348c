"""The block operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only):
``tests/asan/fuzz_block.cpp`` links the C-ABI with stand-ins for the HIP runtime and the launches and
drives it with random descriptors and arguments; the stand-ins check grids and workspace layout."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_epilogue_transformer_tiled_amd", "csrc")
ASAN = os.path.join(ROOT, "tests", "asan")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def fuzzer(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path_factory.mktemp("asan") / "fuzz_block")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
           os.path.join(CSRC, "block_api.cpp"), os.path.join(CSRC, "block_rowwise_api.cpp"),
           os.path.join(ASAN, "fuzz_block.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_fuzz_block_abi(fuzzer, seed):
    r = subprocess.run([fuzzer, str(seed), "20000"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "fuzz ok" in r.stdout and "runtime error" not in r.stderr
