"""A step without sequences asks for a device only where there is a second cursor to write."""
import os

import pytest

from paged_sliding_window_gb300 import binding
from test_fp4_host import FAKE, lib, tables  # noqa: F401


def test_one_cursor_needs_no_device(lib):  # noqa: F811
    assert tables(lib, n=0, pos=FAKE + 64, next=FAKE + 64) == 0


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="host without a GPU only")
def test_two_cursors_need_one(lib):  # noqa: F811
    assert binding.ERRORS[tables(lib, n=0, next=FAKE + 64)] == "PSW_EDEVICE"
