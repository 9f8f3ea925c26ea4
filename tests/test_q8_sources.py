"""A rule of the 8-bit cache's kernels that no result shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_table_gb300", "csrc")


@pytest.mark.parametrize("name", ["decode_attention_q8.cu", "kv_read.cu", "kv_write.cu", "copy_blocks.cu"])
def test_kernels_that_start_early_use_no_read_only_loads(name):
    """These kernels may start while their predecessor writes their inputs.  Loads through
    the read-only path (__ldg, ld.global.nc, const __restrict__ parameters) are for
    data that nothing writes while the kernel lives; griddepcontrol.wait orders the others."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "griddepcontrol.wait" in code
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", code)
