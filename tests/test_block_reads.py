"""What the block operators' buffer loads can reach, on the CPU.

A buffer load's range check covers its vector offset; the scalar offset is defined as excluded from
it, so a distance that the check has to see must not be in the scalar offset.  ``asan/few_reads.cpp`` walks
every lane of the few-row kernels' loads with the address functions that the kernels use."""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_epilogue_transformer_tiled_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def _arguments(text, at):
    """The top-level arguments of the call whose opening parenthesis is at `at`."""
    depth, args, start = 0, [], at + 1
    for i in range(at, len(text)):
        if text[i] in "([{":
            depth += 1
        elif text[i] in ")]}":
            depth -= 1
            if depth == 0:
                return [*args, text[start:i].strip()]
        elif text[i] == "," and depth == 1:
            args.append(text[start:i].strip())
            start = i + 1
    raise AssertionError("unbalanced call")


def test_scalar_offsets_are_zero():
    calls = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        text = open(path).read()
        for m in re.finditer(r"__builtin_amdgcn_raw_(ptr_)?buffer_(load|store)_(\w+)\(", text):
            args = _arguments(text, m.end() - 1)
            # load: resource, offset, scalar offset, policy; store: value first; to LDS: resource, address,
            # size, offset, scalar offset, immediate, policy
            scalar = args[4] if m.group(3) == "lds" else args[3] if m.group(2) == "store" else args[2]
            assert scalar == "0", (os.path.basename(path), text.count("\n", 0, m.start()) + 1, scalar)
            calls += 1
    assert calls > 20


def test_few_row_loads_stay_inside(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path / "few_reads")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                        os.path.join(ROOT, "tests", "asan", "few_reads.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "inside:" in r.stdout, (r.stdout[-1000:], r.stderr[-1000:])
