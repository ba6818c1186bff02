"""The checked build reruns the expert layer's wide cases and those for its accuracy: same results, and no bounds check
fires."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]


def test_checked_build_runs_the_wide_and_the_accurate_cases(cuda):
    if os.environ.get("WQ_LIB") == "checked":
        pytest.skip("already running under the checked build")
    from gemm_wq_gemv_b200 import build
    build.build(checks=True)
    suites = ["tests/test_moe_sizes_gpu.py", "tests/test_moe_accuracy_gpu.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", *suites, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=dict(os.environ, WQ_LIB="checked"), capture_output=True, text=True, timeout=1800)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
