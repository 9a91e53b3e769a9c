import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libq2k")
    config.addinivalue_line("markers", "slow: takes more than a few seconds")
    # Tests without the marker may hand the library addresses that are not the GPU's: a
    # run of those alone sees no GPU, so that no call of theirs can reach one.
    if config.option.markexpr.replace(" ", "") == "notgpu":
        os.environ["CUDA_VISIBLE_DEVICES"] = ""


# Past the argument checks with invented addresses, and refused for want of a device.
NEEDS_NO_GPU = {"test_x_planes_scratch_is_not_needed"}


def pytest_collection_modifyitems(items):
    if os.environ.get("CUDA_VISIBLE_DEVICES") == "" or not os.path.exists("/dev/nvidiactl"):
        return
    for item in items:
        if item.name in NEEDS_NO_GPU:
            item.add_marker(pytest.mark.skip(reason="would launch on invented addresses"))
