"""The numbers by which the bounds-checked build names an access."""
from __future__ import annotations

import collections
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bound_add_gb300", "csrc")


def test_a_number_names_one_source():
    # 700 to 899, which stand for nothing else in these sources
    at = collections.defaultdict(set)
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        name = os.path.basename(path)
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        for n in re.findall(r"\b[78]\d\d\b", code):
            at[int(n)].add(name)
    assert len(at) > 60
    assert not {n: files for n, files in at.items() if len(files) > 1}
