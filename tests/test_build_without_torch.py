"""The C library needs nvcc alone: it is built (here: found up to date) where torch cannot be imported."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc is needed to build the library")

CODE = """
import importlib.util, os, sys
sys.modules["torch"] = None  # import torch raises
spec = importlib.util.spec_from_file_location("_build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
path = b.build()
assert path == b.lib_path() and os.path.exists(path)
print("built", b._binding_fingerprint())
"""


def test_the_library_builds_without_torch():
    from gated_deltanet_linear_delta_gb300 import _build
    _build.build()
    calls = os.stat(_build.calls_path())
    r = subprocess.run([sys.executable, "-c", CODE, _build.__file__], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.split() == ["built", "None"], r.stderr[-2000:]
    # the module for torch tensors that is there stays as it is
    assert os.stat(_build.calls_path()).st_mtime_ns == calls.st_mtime_ns
