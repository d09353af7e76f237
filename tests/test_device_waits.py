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
    # every poll and the end of the limit: no lane returns by itself
    text = source("nm_common.cuh")
    body = re.search(r"bool wait_in_step\([^)]*\) {(.*?)\n}", text, re.S).group(1)
    assert re.search(r"auto complete = \[&\] {\s*return __all_sync\(0xffffffffu, [^;]*\) != 0;\s*};", body)
    assert re.findall(r"if \((.*)\) (?:return true;|{)", body) == [
        "complete()", "complete()", "(++spins & 255u) == 0 && __any_sync(0xffffffffu, global_timer_ns() - t0 > limit)"]
    for name in ("mbar_wait_warp", "mbar_wait_cluster_warp"):
        assert re.search(rf"bool {name}\(uint64_t \*bar, uint32_t parity\) {{\s*return wait_in_step<(true|false)>\(bar, parity\);\s*}}", text)


def test_stream_k_flags_are_taken_by_the_warp():
    # a flag is cleared, and the loop over the later flags ended, on one answer of
    # the warp; the lanes that poll a flag each (k_gemm_wide) vote on all of theirs
    text = source("nm_gemm.cu")
    assert re.findall(r"\bgot = ([^;]*);", text).count("sk_take_flag(flags + (cc * 2 + rank) * 8 + we, seq, lane)") == 1
    assert re.findall(r"(\w+) = sk_wait_flag\(", text) == ["mine"] and "got = __all_sync(0xffffffffu, mine);" in text
    take = re.search(r"bool sk_take_flag\([^)]*\) {(.*?)\n}", source("nm_gemm.cuh"), re.S).group(1)
    assert "__all_sync(0xffffffffu, sk_wait_flag(p, seq))" in take and "__syncwarp" not in take
