"""What the kernels launched beside the one before them may not do, read off their source
(CPU only)."""
import os
import re

import pytest

from hybrid_linear_attention_mixer_b200 import build


def code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return [line.split("//")[0] for line in text.split("\n")]


@pytest.mark.parametrize("name", build.UNITS["serve.cu"])
def test_no_loads_that_need_memory_to_stay_as_it_is(name):
    """The non-coherent path (ld.global.nc, __ldg) is for memory that nothing writes
    while the kernel runs; the kernel before may still write what these read."""
    bad = [line for line in code(name) if re.search(r"__ldg\b|\.nc\b", line)]
    assert not bad, bad
