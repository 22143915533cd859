"""A kernel that overlaps the one before it on the stream waits for that one's end before it touches memory.  The wait may
depend on how the kernel was launched, and not on which work unit comes first: a role that has no part in a CTA's first
unit would never wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_mlp_gb300", "csrc")
CONDITION = re.compile(r"if \(((?:[^()]|\([^()]*\))*)\) \{?\s*pdl_(?:wait|begin)\(\)")
WAITS = [(os.path.basename(path), c) for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
         for c in CONDITION.findall(re.sub(r"//[^\n]*", "", open(path).read()))]


def test_finds_the_waits():
    assert sum(f == "fp8mm.cu" for f, _ in WAITS) >= 4


@pytest.mark.parametrize("file,condition", sorted(set(WAITS)))
def test_waits_depend_on_the_launch_alone(file, condition):
    assert re.fullmatch(r"!?p\.\w+", condition), f"{condition} in {file}"
