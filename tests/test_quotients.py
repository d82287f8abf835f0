"""Numbers of words are split into heads and words by a product in place of a
division: exact over the whole range that paged_read accepts (heads * dim <=
2**24, dim <= 8192)."""

import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_wide_quotients_are_exact(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "quotients")
    r = subprocess.run([nvcc, "-O2", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "bmmc_index_transforms_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "c", "quotients.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_read_splits_its_words_that_way():
    """A product in 32 bits (2**32 / words rounded up) is wrong from 65 heads of
    8191 elements on: the last word of head 64 is taken for one of head 65."""
    words = 8191
    magic = -(-2 ** 32 // words)
    x = 64 * words + words - 1
    assert x * magic >> 32 == 65 and x // words == 64
    with open(os.path.join(ROOT, "bmmc_index_transforms_gb300", "csrc", "paged_cache8.cu")) as f:
        code = f.read()
    kernel = code[code.index("void __launch_bounds__(kReadThreads)"):code.index("bmmc_status launch_read_words")]
    assert "wide_quotient(" in kernel and "__umulhi" not in kernel
