"""What the compiler says of the HIP sources (no GPU is needed)."""
import os
import subprocess

import pytest

from selective_state_space_65_amd import build

SOURCES = build.SRCS + [build.PROBE_SRC]


@pytest.mark.parametrize("source", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_index_is_past_its_array(source):
    """An index that the compiler sees to be past its array, LDS or registers, is a kernel that reads and writes what it does
    not own."""
    r = subprocess.run([build.hipcc()] + build.HIPCC_FLAGS + ["-Werror=array-bounds", "-I", build.INCLUDE, "--cuda-device-only",
                                                              "-fsyntax-only", source], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
