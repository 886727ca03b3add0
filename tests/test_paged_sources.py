"""What the sources of kernels that start while their predecessors run must not do (read on the CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "learned_relative_gqa_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


@pytest.mark.parametrize("name", ["paged_cache.cu", "decode.cu"])
def test_no_non_coherent_loads_in_kernels_launched_early(name):
    """A non-coherent load wants its data unchanged for as long as the kernel runs. These kernels begin
    before the ones that write their inputs end, so what they load is not, whatever they wait for first."""
    text = code(name)
    assert "launch_early(" in text
    assert not re.findall(r"__ldg\s*\(|ld\.global(?:\.\w+)*\.nc|__restrict__", text)


@pytest.mark.parametrize("name", ["paged_cache.cu", "decode.cu"])
def test_every_kernel_launched_early_waits_before_its_first_access(name):
    """Between a kernel's opening brace and its wait there is no access through a pointer of its parameters."""
    kernels = re.split(r"__global__", code(name))[1:]
    assert kernels
    for k in kernels:
        head, _, rest = k[k.index("{"):].partition("wait_for_predecessor();")
        assert rest
        assert not re.search(r"p\.\w+\s*\[|__ld\w+\s*\(|\*\s*reinterpret_cast", head), head
