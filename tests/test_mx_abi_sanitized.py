"""The host-only checks of the 4-bit operators' C ABI (tests/test_mx_abi_cpu.py)
run again against the build instrumented with AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess
import sys

import pytest

from orthogonalising_matrix_optimizer_amd import build_sanitized as bs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_mx_abi_checks_under_address_and_ub_sanitizers():
    bs.build_sanitized()
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_mx_abi_cpu.py")],
                       cwd=ROOT, env=bs.env(), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "passed" in r.stdout
