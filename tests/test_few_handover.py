"""Orders that the kernel of a few tokens relies on are stated in its source (no GPU
needed: what is looked at is the source).

A unit of work waits only for units with lower tickets, and a CTA works on its tickets
in the order in which it holds them; so a CTA has to hold them in ascending order, or
two of them could wait for one another.
"""
import os
import re

import pytest

from tests.test_tensor_memory_rule import CSRC

with open(os.path.join(CSRC, "few.cu")) as f:
    TEXT = re.sub(r"//[^\n]*", "", f.read())


def function(name):
    """Body of a function of few.cu, without comments."""
    start = TEXT.index("{", re.search(r"\b%s\([^;{]*\)\s*{" % name, TEXT).start())
    depth, at = 0, start
    while True:
        depth += {"{": 1, "}": -1}.get(TEXT[at], 0)
        at += 1
        if depth == 0:
            return TEXT[start:at]


def test_one_thread_takes_every_ticket():
    """Atomics of one thread on one address follow its program order; those of several
    lanes of an instruction have no order that CUDA states."""
    body = function("copy_weights")
    takes = re.findall(r"([^;{}]*)atomicAdd\(a\.counters, (\w+)\)", body)
    assert [n for _, n in takes] == ["kAhead", "1"]
    for head, _ in takes:
        assert re.search(r"if \(lane == 0\)|lane == 0 \?", head), head
    assert len(re.findall(r"\bcounters\b", body)) == len(takes)


@pytest.mark.parametrize("role,header", [("copy_rest", "ring.header[s]"), ("multiply", "ring.header[s]"),
                                         ("multiply_scaled", "ring.header[m.at.s]"),
                                         ("finish", "sums.header[buf]")])
def test_a_header_is_read_by_the_whole_warp_before_the_slot_moves_on(role, header):
    """A lane's arrival on a slot's barrier is what lets the slot be used again, its
    header too: the other lanes have read theirs by then."""
    body = function(role)
    read = body.index("const Header h = " + header)
    arrive = re.search(r"\bmbar_arrive\w*\(|\bcp_async_arrive\w*\(", body[read:])
    assert "__syncwarp();" in body[read:read + arrive.start()]


def test_warps_are_whole_at_the_barrier_of_the_lists():
    """bar.sync takes whole warps, whose lanes come from loops of different lengths."""
    body = function("mul_sync")
    assert body.index("__syncwarp();") < body.index("bar.sync")
