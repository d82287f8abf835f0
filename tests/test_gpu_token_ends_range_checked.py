"""The same once more on the bounds-checked build (as
test_gpu_token_ends_checked.py has it for the others)."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ends_of_the_ranges_on_the_bounds_checked_build():
    from bmmc_index_transforms_gb300 import _build

    env = dict(os.environ, BMMC_GB300_LIBRARY=_build.build(checked=True))
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_token_ends_range.py",
           "tests/test_gpu_balance_bits.py"]
    r = subprocess.run(cmd, env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
