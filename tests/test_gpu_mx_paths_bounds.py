"""The paths that only larger microscaled matrices reach, again on the
bounds-checked build (libq4_debug.so), as test_gpu_mx_bounds.py does for the
smaller ones."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mx_paths_on_the_bounds_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_mx_paths.py",
           "tests/test_mx_accuracy.py", "tests/test_mx_workspace.py", "tests/test_mx_empty.py"]
    res = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, Q4_LIBRARY="debug"), capture_output=True, text=True, timeout=900)
    tail = "\n".join((res.stdout + res.stderr).splitlines()[-30:])
    assert res.returncode == 0, tail
    last = tail.splitlines()[-1] if tail else ""
    assert " passed" in last and "skipped" not in last, tail
