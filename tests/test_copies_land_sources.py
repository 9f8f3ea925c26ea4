"""A rule of the decode kernels' loaders that no result shows: no CTA ends while a bulk copy still writes its shared
memory."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_table_gb300", "csrc")


@pytest.mark.parametrize("name,consumers", [("decode_attention_scored.cu", "const int slot = "),
                                            ("decode_attention_q8.cu", "const int slot = "),
                                            ("decode_attention.cu", "const int h = warp;")])
def test_a_loader_waits_for_its_copies_before_every_exit(name, consumers):
    """Consumers that use up their polls leave, so the loader cannot count on their waits: it waits itself where it gives
    up and where it is done, and by a bound that the test hook does not lower."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    at = code.index("auto drain")
    wait = code[at:code.index("};", at)]
    assert "mbar_wait(&full[" in wait and "polls" not in wait
    loader = code[at + len(wait):]
    loader = loader[:loader.index(consumers)]
    # what comes last in the loader: its normal exit
    assert re.search(r"drain\(end - start\);\s*(finish\(\);\s*)?return;\s*\}\s*$", loader)
    assert len(re.findall(r"\bdrain\(", loader)) == 2
