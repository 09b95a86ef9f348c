"""Arguments that the block operators' C-ABI has to refuse or take, under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): ``tests/asan/block_arguments.cpp``."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_epilogue_transformer_tiled_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def test_block_arguments(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path / "block_arguments")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", os.path.join(CSRC, "block_api.cpp"),
           os.path.join(CSRC, "block_rowwise_api.cpp"), os.path.join(ROOT, "tests", "asan", "block_arguments.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "arguments ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
