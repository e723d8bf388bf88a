"""Reads the attention kernels' sources: softmax warps meet at named barriers, which have no limit, so behind
a wait that gave up they must all still take the same segments."""
import os
import re

from fp8_block_scaled_09_b200 import build as fp8bq_build


def source(name):
    with open(os.path.join(fp8bq_build.CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def body(text, head):
    """The braces behind `head`."""
    start = text.index("{", text.index(head))
    depth = 0
    for at in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        if depth == 0:
            return text[start:at + 1]


def test_softmax_warps_of_the_many_row_kernel_take_every_published_segment():
    text = source("attention_many.cuh")
    softmax = text[text.index("setmaxnreg.inc"):text.rindex("__syncthreads()")]
    assert "named_barrier(" in softmax
    loop = body(softmax, "for (;; segs.release())")
    ends = re.findall(r"[^;{}]*\b(?:break|return);", loop)
    # left only where the work list ends; `return` of the nested functions aside
    assert [e.strip() for e in ends if "break" in e] == ["if (sg == nullptr) break;"]
    assert "const Segment *sg = segs.next_published();" in loop and "segs.next(" not in loop
    # which does not depend on when a warp sees the abort flag ...
    taken = body(text, "const Segment *next_published() const")
    assert "abort" not in taken and "*stopped == place(i, phase)" in taken
    # ... and is fixed by the one warp that publishes, when it stops
    work = text[text.index("Items it(a, start_w[0]"):text.index("umma_idesc_e4m3(kHalfRows, kTile)")]
    assert "*seg_stopped = SegReader::place(i, phase);" in body(work, "if (!mbar_wait(&segempty[i], phase ^ 1, abort_flag, status))")


def test_roles_without_named_barriers_leave_as_whole_warps():
    text = source("attention_many.cuh")
    taken = [m.end() for m in re.finditer(r"segs\.next\(abort_flag, status\);", text)]
    assert len(taken) == 3
    for at in taken:
        assert text[at:].lstrip().startswith("if (!__all_sync(0xFFFFFFFFu, sg != nullptr)) break;")


def test_softmax_warps_of_the_few_row_kernel_end_by_the_work_list():
    text = source("attention_few.cuh")
    softmax = text[text.index("float l_run[NR];"):text.rindex("__syncthreads()")]
    loop = body(softmax, "while (cur.next())")
    assert "named_barrier(" in loop and "break;" not in loop and "return;" not in loop


def test_the_query_warp_of_the_few_row_kernel_leaves_as_a_whole():
    """Its loop shuffles with every lane."""
    text = source("attention_few.cuh")
    loop = body(text[text.index("const int sub = lane & 15"):], "while (ok && cur.next())")
    assert "__shfl_xor_sync(0xFFFFFFFFu" in loop
    assert re.findall(r"\bok = [^;]*;", loop) == \
        ["ok = __all_sync(0xFFFFFFFFu, mbar_wait(&qempty[segs & 1], ((segs >> 1) & 1) ^ 1, abort_flag, status));"]
