import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size workloads")


# Their calls name addresses that are made up; some of the solver's pass every check, for the error that a machine without a
# GPU gives at the launch.  The driver is asked, not torch, which may see no GPU where the library does.
MADE_UP_ADDRESSES = {"test_abi_cpu.py", "test_recurrence_abi_cpu.py"}


def driver_has_a_gpu():
    try:
        driver = ctypes.CDLL("libcuda.so.1")
    except OSError:
        return False
    count = ctypes.c_int(0)
    return driver.cuInit(0) == 0 and driver.cuDeviceGetCount(ctypes.byref(count)) == 0 and count.value > 0


@pytest.hookimpl(trylast=True)
def pytest_collection_modifyitems(items):
    named = [item for item in items if item.path.name in MADE_UP_ADDRESSES]
    if named and driver_has_a_gpu():
        for item in named:
            item.add_marker(pytest.mark.skip(reason="a GPU is present: made-up addresses would be used"))


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle
    return oracle.get()
