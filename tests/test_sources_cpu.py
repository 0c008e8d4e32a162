"""Rules that the kernels' sources keep, read from the sources themselves (no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_298_gb300", "csrc")
SOURCES = sorted(sum((glob.glob(os.path.join(CSRC, p)) for p in ("*.cu", "*.cuh", "*.h", "*.cpp")), []))


def code_of(path):
    """The file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_to_several_ctas(path):
    """The library is what every replica of a run on several GPUs loads, and the addresses that its kernels copy from are the
    caller's: no copy is sent to more than one CTA."""
    assert "multicast" not in code_of(path)
