"""What the 4-bit kernels' sources promise and no run can show."""
import os
import re

from paged_sliding_window_gb300 import build


def test_a_warp_has_read_a_part_before_it_is_written():
    """A group's joined part takes the place of its first member. Lanes with the same head read the same
    maximum and sum there, so all have to have read before any writes: lanes of a warp need not run in
    step."""
    text = open(os.path.join(build.CSRC, "fp4_decode.cuh")).read()
    code = re.sub(r"//[^\n]*", "", text)
    joined = re.search(r"add_parts\(from, 1, m\);(.*?)a\.ws_o\[\(slot0 \+ from\)", code, re.S)
    assert joined and "__syncwarp();" in joined.group(1)
