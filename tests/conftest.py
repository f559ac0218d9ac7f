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


def pytest_collection_finish(session):
    gc.collect()
    gc.freeze()  # what is there stays: collections between tests look at what tests make


@pytest.fixture(autouse=True)
def collect_between_gpu_tests(request):
    """GPU tests start without what earlier ones left for the garbage collector: a graph that it destroys during a capture
    ends the capture.  (An exception that a test keeps holds the test's frame, which holds the exception and the test's
    graphs: such rings wait for the collector.)  In them it runs as it does in a user's program."""
    if "gpu" in request.keywords:
        gc.collect()
    yield
