"""How the kernels take a bounded wait that runs out, from their sources.  Each lane of a warp has its
own clock, so lanes may get different answers; a warp that branches on its own lane's answer would meet
barriers, shuffles and votes that its other lanes never reach."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_paged_kv_diag_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["append_kernel.cu", "decode_kernel.cu", "block_bounds.cu", "sparse_attention.cu"])
def test_no_branch_on_one_lanes_answer(name):
    """These kernels leave loops that hold whole-warp operations: the answer is the warp's
    (mbar_wait_warp), or it is kept (`late`) until a vote or a barrier has joined it."""
    code = _code(name)
    assert not re.search(r"\b(if|while|for)\s*\([^;{}]*mbar_wait_bounded\(", code)
    kept = re.findall(r"const bool (\w*late) = !mbar_wait_bounded\(", code)
    assert len(kept) == code.count("mbar_wait_bounded(")
    joined = len(re.findall(r"dead = (?:__any_sync\(kFull, |__syncthreads_or\()\w*late\)", code))
    assert joined == len(kept)


def test_rotating_append_leaves_as_a_whole_block():
    code = _code("rope_append.cu")
    assert re.search(r"landed = mbar_wait_bounded\(.*?if \(__syncthreads_or\(!landed\)\) return;", code, re.S)
    assert code.count("mbar_wait_bounded(") == 2  # (the wait, and the one that lets late copies land)
