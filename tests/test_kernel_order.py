"""The order in which a kernel takes tensor memory and starts, read from the source (on the
GPU a wrong order can only be seen as a hang): a block that took tensor memory while it waits
for the kernel before, or let the kernel behind start before it has its own, can wait for a
block that waits for it, where both fit one multiprocessor."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_group_quantized_qgemv_gb300", "csrc")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for body in text.split("__global__")[1:]:
            if "tc::alloc(" in body:
                yield pytest.param(body, id=os.path.basename(path))


def test_there_are_some():
    assert len(list(kernels())) >= 2


@pytest.mark.parametrize("body", list(kernels()))
def test_tensor_memory_between_the_neighbours(body):
    assert body.count("tc::alloc(") == body.count("pdl_wait()") == body.count("pdl_launch_dependents()") == 1
    assert body.index("pdl_wait()") < body.index("tc::alloc(") < body.index("pdl_launch_dependents()")
    assert body.index("tc::alloc(") < body.index("tc::dealloc(")
