import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200) and the built libmpq.so")
    config.addinivalue_line("markers", "slow: CPU test that takes more than a few seconds")


def pytest_collection_modifyitems(config, items):
    import torch
    if torch.cuda.is_available():
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


@pytest.fixture(autouse=True)
def _no_garbage_while_memory_is_measured(request):
    """A tensor that a caught exception's traceback holds lives in a reference
    cycle until the collector happens to run.  The modules that compare the
    allocated bytes before and after a call start each test without such
    garbage, so that none is freed between their two readings."""
    if "no_alloc" in request.module.__name__:
        gc.collect()
    yield
