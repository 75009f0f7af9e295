"""Copies into shared memory go to one block each (no GPU needed).

A tensor copy that several blocks of a cluster receive is sound for memory of the block's own GPU
alone, and the calls take any device address, so the kernels have none."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_weight_only_gb300", "csrc")


def test_no_copy_has_several_receivers():
    paths = glob.glob(os.path.join(CSRC, "*"))
    assert len(paths) > 10
    copies = 0
    for path in paths:
        with open(path) as f:
            text = f.read()
        # the instruction: a string's pieces, joined, up to its operands
        joined = re.sub(r'"\s*"', "", text)
        for name in re.findall(r"cp\.async\.bulk[\w.:]*", joined):
            copies += 1
            assert "multicast" not in name, (os.path.basename(path), name)
    assert copies >= 3
