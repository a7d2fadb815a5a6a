"""CPU-only: how the kernels of tc_common.cuh use their bounded waits. When a wait's limit runs out while
its phase completes, some lanes of a warp are told so and others are not. The warps go on to
instructions that need all of their lanes, so the answer has to be the warp's: a vote on it. (Making it
happen would need a wait that runs out at a chosen moment, so this reads the source.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_matrix_08_gb300", "csrc")


@pytest.mark.parametrize("name", ["f8_gemm.cu", "orthogonalize.cu"])
def test_warps_leave_their_waits_together(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    statements = [s for s in re.split(r"[;{}]", text) if "wait_short(" in s]
    assert len(statements) >= 4
    for s in statements:
        s = " ".join(s.split())
        # (a wait whose answer nothing depends on: copies that must land before the warp leaves)
        assert re.search(r"__all_sync\(0xffffffffu, .*wait_short\(", s) or s.startswith("wait_short("), s


def test_only_the_first_waits_of_a_product_depend_on_other_blocks():
    """A block without work in a product waits for the next one's operands meanwhile: with the limit of
    the grid-wide barrier, not with that of its own copies."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "orthogonalize.cu")).read())
    voted = [" ".join(s.split()) for s in re.split(r"[;{}]", text) if "__all_sync(" in s]
    first = [s for s in voted if "acc_full" in s or "acc_empty" in s]
    assert len(first) == 2 and all(s.endswith(", limit))") for s in first), first
    assert len(re.findall(r"limit = kWaitLimitNs;", text)) == 2
