"""The microscaled and expert-routing tests again on the bounds-checked build
(libq4_debug.so), in a child process as test_gpu_bounds.py does it: the
outputs are compared as usual, and conftest asserts after each test that no
kernel met an index outside its buffer."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mx_on_the_bounds_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_mx.py", "tests/test_gpu_experts.py"]
    res = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, Q4_LIBRARY="debug"), capture_output=True, text=True,
                         timeout=900)
    tail = "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    assert res.returncode == 0, tail
    last = tail.splitlines()[-1] if tail else ""
    assert " passed" in last and "skipped" not in last, tail
