import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def collect_between_gpu_tests(request):
    """The garbage collector runs between GPU tests, not in them: a graph of an earlier test that it destroys during a
    capture ends the capture.  (An exception that a test keeps holds the test's frame, which holds the exception and
    the test's graphs: such rings wait for the collector.)"""
    if "gpu" not in request.keywords:
        yield
        return
    gc.disable()
    yield
    gc.enable()
    gc.collect(0)
