import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: takes more than a few seconds")


# Modules that call the library with made-up addresses: without a device every
# such call is refused; with one, those whose other arguments are right would run.
NO_DEVICE_ONLY = {"test_window_host.py"}


def skip_made_up_addresses(items, has_gpu):
    if has_gpu:
        for item in items:
            if os.path.basename(str(item.path)) in NO_DEVICE_ONLY:
                item.add_marker(pytest.mark.skip(reason="made-up addresses: only where there is no device"))


def pytest_collection_modifyitems(config, items):
    import torch

    skip_made_up_addresses(items, torch.cuda.is_available())


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle.oracle as o

    return o.load_library()
