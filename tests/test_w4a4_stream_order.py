"""The order of what the kernels on 4-bit activations read and whom they launch (no GPU needed).

A kernel that is launched while the one in front of it still runs may not copy anything before
griddepcontrol.wait, since that kernel may be what writes it, and launches the next one only behind
it: a decode product behind it reads its weight at once and counts on what is in front of this
kernel to be finished."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_weight_only_gb300", "csrc")


def kernels(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for part in re.split(r"__global__", text)[1:]:
        body = part[:part.index("\n}\n")]
        if "griddepcontrol" in body:
            yield re.search(r"(\w+_kernel)\(", body).group(1), body


@pytest.mark.parametrize("name,count", [("w4a4_gemm.cu", 2), ("w4a4_rows.cu", 2), ("experts.cu", 5)])
def test_kernels_wait_before_they_copy_and_before_they_launch_the_next(name, count):
    seen = list(kernels(name))
    assert len(seen) == count
    for kernel, body in seen:
        waits = [m.start() for m in re.finditer(r"griddepcontrol\.wait", body)]
        launches = [m.start() for m in re.finditer(r"griddepcontrol\.launch_dependents", body)]
        copies = [m.start() for m in re.finditer(r"bulk_copy_g2s|copy_box\(", body)]
        assert len(launches) == 1 and launches[0] > max(waits), kernel
        assert all(at > max(waits) for at in copies), kernel
