"""Host tests that hand the library valid calls on made-up addresses, to see
which of its checks they pass, are not run on a machine with a GPU."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.no_gpu
def test_says_what_it_is():
    pass


def _outcome(tmp_path, test, present):
    """How a run ends on a machine that says whether it has a GPU.  (The tests
    named here are chosen by their marks alone: nothing of theirs is run where
    there really is one.)"""
    (tmp_path / "claims.py").write_text(f"import torch\ntorch.cuda.is_available = lambda: {present}\n")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-p", "claims", test], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.strip().splitlines()[-1]


def test_kept_off(tmp_path):
    line = _outcome(tmp_path, "tests/test_addresses_only.py::test_says_what_it_is", True)
    assert "1 skipped" in line and "passed" not in line


def test_run_without(tmp_path):
    line = _outcome(tmp_path, "tests/test_addresses_only.py::test_says_what_it_is", False)
    assert "1 passed" in line


@pytest.mark.no_gpu
@pytest.mark.parametrize("test", ["tests/test_token_moves_host.py::test_slices_of_one_array_are_told_apart"])
def test_those_without_the_mark(tmp_path, test):
    assert "1 skipped" in _outcome(tmp_path, test, True)
