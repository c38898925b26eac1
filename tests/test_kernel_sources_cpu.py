"""What the kernels' sources have to keep to, read as text."""
import os
import re

import pytest

from depth_wise_attention_attnres_gb300 import build

FILES = [os.path.join(build.CSRC, name) for name in build.SOURCES + build.HEADERS]


def code(path):
    """A source without its comments."""
    with open(path) as fh:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", fh.read(), flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_no_loads_through_the_read_only_path(path):
    """Kernels are launched with programmatic serialization and so may start while the kernel before them still writes
    what they read. Loads through the read-only path are promised correct only for memory nobody writes during a
    kernel's life, and may be moved ahead of the wait for that kernel: neither they nor the qualifier that lets the
    compiler choose them are used."""
    found = re.findall(r"__ldg\b|\bld\.global(?:\.\w+)*\.nc\b|__restrict__", code(path))
    assert not found, found
