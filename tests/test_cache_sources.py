"""Rules that the cache operators' kernels keep in their sources; no GPU."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_command_execution_gb300", "csrc")


def test_no_read_only_loads():
    """The kernels begin while the previous one on their stream still runs, and read what it writes (a selection's
    tables, an append's pages). Loads through the read-only path are for memory that nothing writes while the kernel
    lives: they are neither ordered after the wait for the previous kernel nor coherent."""
    files = [f for f in glob.glob(os.path.join(CSRC, "cache_*.cu*"))]
    assert len(files) >= 6
    for f in files:
        with open(f) as src:
            text = re.sub(r"//[^\n]*", "", src.read())
        if "wait_for_previous" in text or f.endswith(".cuh"):
            assert not re.search(r"__ldg\b|\.nc\b|__restrict__", text), os.path.basename(f)
