"""The refusals, planners and workspace sizes of the distillation and norm
calls under the host AddressSanitizer and UndefinedBehaviorSanitizer build:
tests/test_abi_ops.py against it in a child process."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_abi_of_the_operators_under_asan_and_ubsan():
    sys.path.insert(0, ROOT)
    from cross_entropy_amd import build as b
    try:
        b.build(sanitize=True)
    except RuntimeError as e:   # pragma: no cover
        pytest.fail(f"sanitizer build failed: {e}")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_ops.py")],
                       env=b.sanitizer_env(), capture_output=True, text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr
