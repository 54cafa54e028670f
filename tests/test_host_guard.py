"""Host checks with made-up addresses never run where a device would take them."""
import os
import re

from tests import conftest


class Item:
    def __init__(self, path):
        self.path, self.marks = path, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_made_up_addresses_are_skipped_beside_a_device():
    items = [Item("/x/tests/test_window_host.py"), Item("/x/tests/test_gpu_window_attn.py")]
    conftest.skip_made_up_addresses(items, has_gpu=False)
    assert not items[0].marks and not items[1].marks
    conftest.skip_made_up_addresses(items, has_gpu=True)
    assert items[0].marks == ["skip"] and not items[1].marks


def test_modules_with_made_up_addresses_are_known():
    """Those of the window and cache entry points; the dilated ones' skip such calls themselves."""
    here = os.path.dirname(os.path.abspath(__file__))
    found = {f for f in os.listdir(here) if f.endswith(".py") and f != os.path.basename(__file__)
             and re.search(r"c_void_p\(0x|=0x1000", open(os.path.join(here, f)).read())}
    assert found - {"test_abi_cpu.py"} <= conftest.NO_DEVICE_ONLY
