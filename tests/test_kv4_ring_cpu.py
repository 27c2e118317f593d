"""The order of the rows kernel's ring in shared memory, read from its source.

A warp's stage is filled by the cp.async copies of all its lanes and read by all of them, and cp.async.wait_group covers
the copies of the lane that executes it alone.  So every turn of the loop needs a barrier of the warp between the wait and the first
read (the others' copies have arrived), and one between the last read and the next copies into that stage (the others have
read).  Nothing but the order of the source shows that: a warp whose lanes happen to run together gives right results without."""
import os
import re

import ternary_weight_bit_b200 as tb

SOURCE = os.path.join(os.path.dirname(tb.__file__), "csrc", "kv4_attention.cu")


def events():
    """The ring's operations in one turn of the tile loop, in the order of the source."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    start = text.index("for (int it = 0; it < count; ++it)")
    depth, end = 0, start
    for end in range(text.index("{", start), len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            break
    kinds = {"fetch(": "copy", "copies_wait<": "wait", "take<": "read", "__syncwarp(": "barrier"}
    return [kinds[m] for m in re.findall(r"fetch\(|copies_wait<|take<|__syncwarp\(", text[start:end])]


def test_each_turn_of_the_ring_has_its_two_barriers():
    turn = events()
    assert turn.count("copy") == 1 and turn.count("wait") == 1 and turn.count("read") >= 4
    twice = turn + turn  # this turn's last reads are followed by the next turn's copies
    for i, e in enumerate(twice):
        if e == "wait":
            after = twice[i + 1:]
            assert "read" not in after or "barrier" in after[:after.index("read")], "a read before the others' copies are there"
        if e == "copy" and "read" in twice[:i]:
            before = twice[:i]
            last = len(before) - 1 - before[::-1].index("read")
            assert "barrier" in before[last:], "a copy over what others may still read"
