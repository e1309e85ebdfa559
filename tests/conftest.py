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
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) and the built HIP library")
    config.addinivalue_line("markers", "slow: large inputs; minutes of CPU time")


# Files whose `lib` tests hand the C ABI addresses that are no memory. A call that passes validation there is stopped by
# the device check alone, so on a host with a GPU it would launch a kernel that reads or writes them.
PLACEHOLDER_POINTER_FILES = ("test_abi_cpu.py", "test_operators_abi_cpu.py")


def pytest_collection_modifyitems(config, items):
    import torch

    if not torch.cuda.is_available():
        return
    skip = pytest.mark.skip(reason="placeholder pointers: host without a GPU only")
    for item in items:
        if os.path.basename(str(item.fspath)) in PLACEHOLDER_POINTER_FILES and "lib" in getattr(item, "fixturenames", ()):
            item.add_marker(skip)
