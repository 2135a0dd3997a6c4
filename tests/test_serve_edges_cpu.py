"""The decode-step operators where their tests on a GPU cannot show a fault (no GPU needed)."""
import glob
import os
import re

import pytest

from latency_barrier_free_gb300 import build_ext

torch = pytest.importorskip("torch")


def source(name):
    text = open(name).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_operator_reads_through_the_non_coherent_path():
    """A grid that is launched before its predecessor has ended may hold on to what that path read of a buffer; the operators
    read each other's results."""
    names = glob.glob(os.path.join(build_ext.CSRC, "serve*.cu*"))
    assert len(names) >= 6
    for name in names:
        text = source(name)
        for word in ("__ldg(", "ld.global.nc", "ld_nc", "__restrict__"):
            assert word not in text, (name, word)
