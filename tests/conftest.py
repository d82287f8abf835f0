import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")
    config.addinivalue_line("markers", "no_gpu: hands the library valid calls on addresses that are only looked at; "
                                       "not run where there is a GPU, which would launch them")


# Tests of that kind without the mark.  (Where the GPU reads pageable memory,
# as on a Grace host, any address passes the library's check of the pointers.)
LOOKED_AT = {"test_token_moves_host.py": {"test_slices_of_one_array_are_told_apart"}}


def pytest_collection_modifyitems(items):
    kept_off = [x for x in items if x.get_closest_marker("no_gpu")
                or getattr(x, "originalname", x.name) in LOOKED_AT.get(x.path.name, ())]
    if not kept_off:
        return
    try:
        import torch

        present = torch.cuda.is_available()
    except ImportError:
        present = os.path.exists("/dev/nvidiactl")
    for x in kept_off if present else ():
        x.add_marker(pytest.mark.skip(reason="its calls would be launched"))


GOLDEN = os.path.join(ROOT, "tests", "golden")


def read_golden(name):
    """Rows of a whitespace-separated golden file, comments stripped."""
    rows = []
    with open(os.path.join(GOLDEN, name)) as f:
        for line in f:
            line = line.split("#", 1)[0].strip()
            if line:
                rows.append(line.split())
    return rows


@pytest.fixture(scope="session")
def golden():
    return read_golden


@pytest.fixture(autouse=True)
def _bounds_record_stays_clean(request):
    """When the bounds-checked build of the library is the one loaded (its
    path in BMMC_GB300_LIBRARY), every GPU test must leave the device-side
    failure record empty: no kernel access outside its buffers or shared
    arrays."""
    if not os.environ.get("BMMC_GB300_LIBRARY") or request.node.get_closest_marker("gpu") is None:
        yield
        return
    from bmmc_index_transforms_gb300 import _capi

    L = _capi.lib()
    r = _capi.BoundsReport()
    assert L.bmmc_bounds_report(ctypes.byref(r), 1) == _capi.OK
    assert r.enabled == 1, "BMMC_GB300_LIBRARY does not name a bounds-checked build"
    yield
    assert L.bmmc_bounds_report(ctypes.byref(r), 1) == _capi.OK
    assert r.failures == 0, (f"{r.failures} kernel accesses outside their buffers; first at site {r.site} "
                             f"(file tag * 100000 + line), address {r.address:#x}, {r.bytes} bytes, "
                             f"range [{r.lo:#x}, {r.hi:#x})")
