"""Static checks on the CUDA sources (CPU): how the products' roles wait and give up."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_block_scaled_07_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_roles_wait_as_whole_warps():
    """Each role of the products is a warp that goes on to warp-wide instructions (elect.sync, tcgen05.ld): a wait that
    answers lane by lane could, once one has run out, send some of its lanes on and others to the exit."""
    for name in ("gemm.cuh", "gemm_few.cuh"):
        text = code(name)
        assert "mbar_wait_warp(" in text
        assert not re.search(r"\bmbar_wait\(", text), f"{name}: a wait that answers lane by lane"
