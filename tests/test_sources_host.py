"""Every CUDA source is reached: .cu files are in the directory that the build compiles (or are a host test's), headers are included by one of them."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_weight_only_sgemv_gb300", "csrc")
HOST = os.path.join(ROOT, "tests", "host")


def _sources():
    """The repository's CUDA sources (what git ignores left out)."""
    ignored = {os.path.join(ROOT, line.strip().strip("/")) for line in open(os.path.join(ROOT, ".gitignore")) if line.strip().endswith("/")}
    for at, dirs, files in os.walk(ROOT):
        dirs[:] = [d for d in dirs if not d.startswith((".", "_")) and os.path.join(at, d) not in ignored]
        for f in files:
            if f.endswith((".cu", ".cuh")):
                yield os.path.join(at, f)


def test_sources_are_where_they_are_built():
    assert {os.path.dirname(f) for f in _sources()} <= {CSRC, HOST}


def test_headers_are_included():
    names = [f for f in _sources() if f.endswith(".cuh")]
    used = set()
    for f in _sources():
        used |= {os.path.basename(x) for x in re.findall(r'#include "([^"]+)"', open(f).read())}
    assert names and not [f for f in names if os.path.basename(f) not in used]
