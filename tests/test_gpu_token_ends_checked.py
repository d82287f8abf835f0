"""The GPU tests of embeddings, the balance loss and 8-bit caches, and of the
decoder that runs them, once more on the bounds-checked build: every global
access of their kernels lies inside the arrays that the call describes, every
shared access inside the kernel's arrays, and after every test the record of
failed accesses is empty (tests/conftest.py)."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_token_ends_on_the_bounds_checked_build():
    from bmmc_index_transforms_gb300 import _build

    env = dict(os.environ, BMMC_GB300_LIBRARY=_build.build(checked=True))
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_embedding.py",
           "tests/test_gpu_balance.py", "tests/test_gpu_paged_cache8.py", "tests/test_gpu_token_model.py"]
    r = subprocess.run(cmd, env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
    print(r.stdout.strip().splitlines()[-1])
