"""A kernel that is launched early starts while the one before it still writes
what it is going to read.  Read-only loads (of a __restrict__ const parameter, or
__ldg) promise that nothing writes for as long as the kernel lives, so the compiler may
move them ahead of the wait, or serve them from a cache that is not told of
the writes: such a kernel reads only the caller's arrays that way.  Read from
the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bmmc_index_transforms_gb300", "csrc")
CALLERS = {"ids", "grad", "logits"}  # ready before the call's first kernel starts
WAIT = "cudaGridDependencySynchronize()"


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _kernels(code):
    """(name, parameters, body) of the kernels."""
    for part in re.split(r"__global__", code)[1:]:
        m = re.match(r"\s+void\s+(?:__launch_bounds__\([^;{]*?\)\s+)?(\w+)\(", part)
        if m:
            body = part.index("{")
            end = part.find("\n}\n", body)
            yield m.group(1), part[m.end():body], part[body:end]


def _waiting():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            for kernel, parameters, body in _kernels(_code(name)):
                if WAIT in body:
                    yield name, kernel, parameters, body


def test_every_wait_is_found():
    found = [k for _, k, _, _ in _waiting()]
    assert len(found) == sum(_code(n).count(WAIT) for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")))
    assert {"sort_place_kernel", "digit_count_kernel", "digit_place_kernel", "sum_rows_kernel", "join_parts_kernel",
            "balance_join_kernel"} <= set(found)


@pytest.mark.parametrize("name,kernel,parameters,body", list(_waiting()), ids=lambda x: x if x.isidentifier() else "")
def test_nothing_that_is_being_written_is_read_only(name, kernel, parameters, body):
    for constant in re.findall(r"const \w+\s*\* __restrict__ (\w+)", parameters):
        assert constant in CALLERS, f"{name}: {kernel} reads {constant} as if nothing wrote it"
    assert "__ldg(" not in body
