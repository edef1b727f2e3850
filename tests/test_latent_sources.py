"""What the latent kernels' sources promise and no run can show."""
import os
import re

from paged_sliding_window_gb300 import build


def test_dependent_launches_read_coherently():
    """Kernels that are launched while what is ahead of them still runs may be alive while their
    inputs are written. The read-only path is for data that does not change during a kernel's
    life: no __ldg and no const __restrict__ input in a source that launches so."""
    found = 0
    for name in build.SOURCES:
        text = open(os.path.join(build.CSRC, name)).read()
        code = re.sub(r"//[^\n]*", "", text)
        if "griddepcontrol.wait" not in code:
            continue
        found += 1
        assert "__ldg" not in code, name
        assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", code), name
    assert found == 1
