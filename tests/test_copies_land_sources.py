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


@pytest.mark.parametrize("name", ["prefill_tc.cu", "decode_attention_shared.cu"])
def test_threads_that_issue_mmas_wait_for_them_before_every_exit(name):
    """Softmax warps that use up their polls do not wait for the last S, so its issuing thread always does; the PV thread
    waits for its last commit, or where it gives up for all it issued."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert len(re.findall(r"\}\s*land\(0\);\s*\}\s*__syncwarp\(\);", code)) == 1
    assert len(re.findall(r"mbar_wait\(&sm->kv_empty\[[^;]*\) fail = true;\s*if \(fail\) land\(1\);\s*\}\s*__syncwarp\(\);", code)) == 1
    land = code[code.index("auto land"):]
    land = land[:land.index("};")]
    assert "tc_commit(&sm->last[i])" in land and "polls" not in land
