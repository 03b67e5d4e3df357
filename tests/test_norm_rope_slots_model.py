"""Order of the shared-memory slots in the norm's backward from 8-bit rows
(csrc/qk_norm_rope.cu), on the CPU.  The first thread of a row copies the row's
scale into its slot asynchronously, and kDepth steps later the same slot is copied
into again.  A thread that reads its own slot alone needs no more than the order
of its own copy, wait and read.  Where other threads read the slot, only
__syncwarp() orders memory between them (shuffles make them meet, but order
nothing, and a load may be carried out any time before the next fence), so with
the fences of the loop as the source has them:
  the wait for a step's copies lies in an earlier interval than the step's reads,
  a step's reads lie in an earlier interval than the next copy into their slot.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_block_sparse_pool_b200", "csrc")


def block(text, start):
    """The braces' content that begins behind `start`."""
    i = text.index("{", text.index(start) + len(start) - 1)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i + 1:j]
    raise AssertionError(start)


def program():
    """One step of the loop, as the source has it for codes: fence, copy, wait, read."""
    src = re.sub(r"//.*", "", open(os.path.join(CSRC, "qk_norm_rope.cu")).read())
    depth = int(re.search(r"kDepth = (\d+);", src).group(1))
    kernel = block(src, "qk_norm_rope_bwd_kernel(const BwdArgs<TX, TG> a) {")
    loop = block(kernel, "for (int h = ha + slot; h - slot < hz; h += RPW) {")
    read = block(src, "read_slot(const uint4* slot, Raw<int8_t>& r, int sub) {")
    ops = []
    token = r"(__syncwarp\(\))|(fetch_step\(\))|(copy_wait<)|(read_slot\(from, raw)"
    for m in re.finditer(token, loop):
        if m.group(4):
            ops += ["fence"] * read[:read.index("r.scale")].count("__syncwarp()") + ["read"]
            ops += ["fence"] * read[read.index("r.scale"):].count("__syncwarp()")
        else:
            ops.append("fence" if m.group(1) else "copy" if m.group(2) else "wait")
    assert ops.count("copy") == ops.count("wait") == ops.count("read") == 1
    return ops, depth, "slot - sub" in read  # the last: other threads' slots are read


def races(ops, depth, steps=20):
    interval, t = 0, {}
    for i in range(depth - 1):
        t["copy", i] = 0                            # ahead of the loop
    for i in range(steps):
        for op in ops:
            if op == "fence":
                interval += 1
            else:
                t[op, i + depth - 1 if op == "copy" else i] = interval
    found = []
    for i in range(steps):
        if not t["wait", i] < t["read", i]:
            found.append("read before the copy has landed")
        if ("copy", i + depth) in t and not t["read", i] < t["copy", i + depth]:
            found.append("copied into while it may still be read")
    return found


def test_the_loop_of_the_source():
    ops, depth, others = program()
    if others:
        assert races(ops, depth) == []
    else:  # each thread for itself; what is read goes to the row's threads by a shuffle
        assert [op for op in ops if op != "fence"] == ["copy", "wait", "read"]


@pytest.mark.parametrize("ops,what", [
    (["copy", "wait", "fence", "read"], "copied into while it may still be read"),
    (["fence", "copy", "wait", "read"], "read before the copy has landed"),
    (["fence", "copy", "fence", "wait", "read"], "read before the copy has landed"),
])
def test_missing_fences_are_caught(ops, what):
    assert what in races(ops, 4)


def test_fences_on_both_sides_hold():
    assert races(["fence", "copy", "wait", "fence", "read"], 4) == []
