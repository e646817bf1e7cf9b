"""Rules of the target-side calls that show without a GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_hf_gb300", "csrc")
TARGET = ["attn.cuh", "attn_rows.cu", "attn_tc.cu", "pages.cu", "pages.cuh", "verify.cu"]


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        s = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


@pytest.mark.parametrize("name", TARGET)
def test_what_an_earlier_call_may_still_write_is_read_coherently(name):
    """The kernels start while the launch before them runs, which may write any of their inputs: lengths, tables,
    drafts, logits, rows. The non-coherent path is for data that nobody writes while the kernel lives."""
    code = _code(name)
    assert "__ldg(" not in code and "ld.global.nc" not in code and "__restrict__" not in code


def test_warps_are_together_where_an_instruction_wants_them():
    """tcgen05.ld and setmaxnreg are executed by a whole warp: behind code that lanes leave apart (a loop whose
    length goes by the lane, a `continue` of some) a __syncwarp() comes first."""
    code = _code("attn_tc.cu")
    kernel = code[code.index("tc_kernel("):]
    before = kernel[:kernel.index('"setmaxnreg')]
    assert re.search(r"check_offsets\(a, tid, TCT\);\s*__syncwarp\(\);", before)
    loops = re.split(r"for \(int q = 0; q < DH; q \+= 32\) \{", kernel)[1:]
    assert len(loops) == 2
    assert "continue" not in loops[0][:loops[0].index("tmem_st32")]  # the rescaling: no lane leaves it
    assert "if (!valid) continue;" in loops[1] and re.match(r"\s*__syncwarp\(\);", loops[1])


def test_nothing_is_in_flight_when_a_cta_gives_up():
    """Behind a wait that ran out: the products issued are waited for (one commit behind them all) before TMEM is
    given back and the CTA ends, as the copies are."""
    code = _code("attn_tc.cu")
    tail = code[code.rindex("if (*abort_flag) {"):code.index("if (warp == 1) tmem_dealloc")]
    assert re.search(r"mma_commit\(elect_one\(\), smem_u32\(drained\)\);\s*wait_uniform\(smem_u32\(drained\), 0\);", tail)
    assert tail.count("mbar_wait(") == 2 and tail.rstrip().endswith("tc_fence_after();")
    assert "mbar_init(drained, 1)" in code


def test_the_bounds_of_prompts_are_checked_whoever_takes_the_first_item():
    """Items are the launch's CTAs, and one that has not started can be taken over by another: also the first, whose
    work includes the look at the bounds."""
    code = _code("attn_tc.cu")
    loop = code[code.index("take_next_cta(answer, n_full);"):]
    assert re.search(r"idx = came \? taken_cta\(answer\) : -1;.*?if \(idx == 0\) check_offsets\(a, lane, 32\);", loop, re.S)
