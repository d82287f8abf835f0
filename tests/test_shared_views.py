"""In the bounds-checked build the token moves' kernels test every access of
their shared arrays against that array's own length: they have no other way to
an element than the views that make the test (Slots in token_words.cuh).  Read
from the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bmmc_index_transforms_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        s = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", s, flags=re.S))


def _statements(code):
    return [" ".join(x.split()) for x in re.split(r"[;{}]", code)]


@pytest.mark.parametrize("name,arrays", [("experts.cu", 10), ("rotary.cu", 5)])
def test_shared_arrays_are_reached_through_views(name, arrays):
    code = _code(name)
    # a struct of arrays is reached by its members
    members = [(m.group(2), re.findall(r"(\w+)\[\w+\]", m.group(1)))
               for m in re.finditer(r"__shared__ struct \{(.*?)\} (\w+)\[", code, flags=re.S)]
    names = re.findall(r"__shared__ (?!struct)(?:const )?\w+\*? (?:const )?(\w+)\[", code)
    assert len(names) + sum(len(m) for _, m in members) >= arrays, (names, members)
    for s in _statements(code):
        allowed = "__shared__" in s or "BMMC_SPANS_ENTER" in s or re.match(r"const Slots<[^=]*> \w+\(", s)
        if allowed:
            continue
        for n in names:
            assert not re.search(rf"\b{n}\b", s), f"{name}: {n} without a view: {s}"
        for outer, inner in members:
            for m in inner:
                assert f"mine.{m}" not in s, f"{name}: {outer}.{m} without a view: {s}"
    # a view's pointer is used where its test stands in front of it, or to lay another view beside it
    for line in code.splitlines():
        for _ in re.finditer(r"\b(\w+)\.p\b", line):
            assert ".ok(" in line or "const Slots<" in line or "__cvta_generic_to_shared(words.p + to)" in line, line


def test_a_view_gives_no_element_without_the_test():
    code = _code("token_words.cuh")
    view = code[code.index("struct Slots"):code.index("template <int BYTES> struct WordOf;")]
    assert "operator" not in view
    checked = view[view.index("#ifdef BMMC_BOUNDS_CHECK"):view.index("#else")]
    for line in checked.splitlines():
        if "p[i]" in line or "atomicAdd" in line:
            assert "ok(i, line)" in line, line
