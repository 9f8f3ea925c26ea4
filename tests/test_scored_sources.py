"""A rule of the kernels behind changed scores and shared prefixes that no result shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_table_gb300", "csrc")


@pytest.mark.parametrize("name", ["decode_attention_scored.cu", "decode_attention_shared.cu"])
def test_kernels_that_start_early_use_no_read_only_loads(name):
    """These kernels may start while their predecessor writes their inputs: no loads through the read-only path."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "griddepcontrol.wait" in code
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", code)


def test_prefill_uses_no_read_only_loads():
    test_kernels_that_start_early_use_no_read_only_loads("prefill_tc.cu")
