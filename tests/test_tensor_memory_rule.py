"""Tensor memory is never held across a wait for a CTA that may be waiting for
tensor memory (no GPU needed: what is looked at is the order in the source).

tcgen05.alloc has no time limit.  A cta_group::1 kernel that waits for its cluster
while it holds columns can meet another such kernel, of another stream, on two SMs
in opposite orders, and neither ends.  (The cta_group::2 kernels, which cannot do
without their peer, are kept off one another's SMs by their shared memory, which
static_asserts hold.)
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_routed_expert_fp32_gb300", "csrc")


def kernels(path):
    """(name, body) of every __global__ function in the file, without comments."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        depth, at = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        head = text[m.end():start]
        yield re.findall(r"(\w+_kernel)\b", head)[0], text[start:at]


ALL = [(os.path.basename(p), name, body) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
       for name, body in kernels(p)]
ONE = [k for k in ALL if re.search(r"\btmem_alloc\(", k[2])]


def test_the_kernels_are_found():
    assert {"adapter_shrink_tile_kernel", "adapter_split_kernel", "gemm_tc_kernel"} <= \
        {name for _, name, _ in ONE}


def test_ctas_of_two_pair_kernels_never_meet_on_an_sm():
    """Those of the experts' pair kernel take more than half of an SM's shared memory
    (the adapter projection's, by a static_assert, too)."""
    pairs = {file for file, _, body in ALL if "tmem_alloc_pair(" in body}
    assert pairs == {"ffn_tc2.cu", "adapter_tile.cu"}
    with open(os.path.join(CSRC, "ffn_tc2.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    value = {}
    for name, expr in re.findall(r"constexpr int (kP\w+) = ([^;]+);", text):
        value[name] = eval(expr.replace("/", "//"), {}, value)
    assert 2 * (value["kPSmem"] + 1024) > 228 * 1024
    with open(os.path.join(CSRC, "adapter_tile.cu")) as f:
        assert "static_assert(fills_half_sm(kSmem)" in f.read()


@pytest.mark.parametrize("file,name,body", ONE, ids=[k[1] for k in ONE])
def test_tensor_memory_is_freed_before_the_cluster_is_waited_for(file, name, body):
    alloc = body.index("tmem_alloc(")
    free = body.index("tmem_dealloc(", alloc)
    between = body[alloc:free]
    for wait in ("cluster_sync_all", "grid_wait"):
        assert wait not in between, f"{file}: {name} holds tensor memory in {wait}"
