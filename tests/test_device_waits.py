"""Host-side reading of the kernels' bounded waits (no GPU needed; a wait that
runs out in the middle of a kernel cannot be staged without leaving copies in
flight).  Each lane of a warp measures a wait's limit by itself, so a warp whose
lanes run a loop together has to agree on the outcome before it goes on: a lane
that left the loop alone would be missing at the next warp-wide instruction, for
which the others wait without a limit."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_structured_sparse_diag_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["nm_ffn.cu", "nm_grad.cu"])
def test_warps_in_step_wait_together(name):
    # the loading, issuing and epilogue warps of these files all run in step
    text = source(name)
    assert re.search(r"\bmbar_wait(_cluster)?_warp\(", text)
    assert not re.findall(r"[^\n]*\bmbar_wait(?:_cluster)?\([^\n]*", text)


def test_a_common_wait_is_a_vote():
    text = source("nm_common.cuh")
    for name in ("mbar_wait", "mbar_wait_cluster"):
        body = re.search(rf"bool {name}_warp\([^)]*\) {{(.*?)}}", text, re.S).group(1)
        assert re.fullmatch(rf"\s*return __all_sync\(0xffffffffu, {name}\(bar, parity\)\);\s*", body)
