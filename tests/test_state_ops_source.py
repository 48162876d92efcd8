"""What no input reaches without a fault: a wait inside the 8-bit AdamW kernel
that gives up, and a device flag that another kernel raises meanwhile.  The
kernels' source is read instead.

Blocks of 256 elements are reduced over a whole warp (shuffles and maxima that
name all 32 lanes), so whether a warp goes on has to be one answer for its
lanes, formed by a vote."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "matrix_aware_optimizer_step_b200",
                    "csrc")


def source():
    with open(os.path.join(CSRC, "state_ops.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(name):
    """The braces of the function `name`, without comments."""
    text = source()
    at = text.index("{", re.search(r"\b" + name + r"\([^;{]*\)\s*\{", text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(name)


VOTE = r"__(?:all|any)_sync\(0xffffffffu,"


def test_a_warp_takes_one_answer_from_its_wait():
    """Each lane polls by its own clock: the lanes' answers are put together
    before the kernel acts on them."""
    assert re.search(VOTE + r"\s*lane_wait\(", body("bulk_wait"))
    kernel = body("adamw8_kernel")
    assert "bulk_wait(" in kernel and "lane_wait(" not in kernel


def test_a_warp_takes_one_answer_from_the_flags_and_scalars():
    assert re.search(r"d\.go = " + VOTE, body("adam_now"))
    assert re.search(VOTE + r"\s*halted\(flags\)\)", body("state8_kernel"))


def test_a_wait_that_gives_up_leaves_no_codes_without_their_scales():
    """Tails store their codes before the wait; their scales have to follow
    on every way out, those of blocks that were not stepped stay."""
    kernel = body("adamw8_kernel")
    wait = kernel.index("bulk_wait(")
    tail, loop = kernel.index("STOCH, false>"), kernel.index("STOCH, true>")
    assert tail < wait < loop
    gave_up = kernel[wait:loop]
    at = gave_up.index("store_scales(whole)")       # ahead of the return that the failed wait takes
    assert at < gave_up.index("return", at) and "return" not in gave_up[:at].replace("if (!now.go) return;", "")
    assert "store_scales(0)" in kernel[loop:]
