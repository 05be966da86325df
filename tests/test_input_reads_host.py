"""Source check: kernels that may be resident while the grid before them writes (programmatic launch) read nothing by
a load that is defined only for data constant during the kernel."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_kv_cache_fp8kv_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_no_read_only_loads(path):
    code = _code(path)
    assert not re.search(r"__ldg\b|\.nc\b", code)
    assert not re.search(r"\bconst\s+\w+\s*\*\s*__restrict__", code)


def test_every_programmatic_launch_waits():
    """A file whose launches may start early has kernels that wait for the grid before them."""
    for path in FILES:
        if path.endswith(".cu") and "ProgrammaticStreamSerialization" in _code(path):
            assert "griddep_wait()" in _code(path), path
