"""Shared memory that one CTA writes and the other CTA's MMAs read is handed over at
cluster scope (no GPU needed: what is looked at is the source).

In the pair kernel of the adapter projection the low-rank operands are plain writes of
both CTAs and rank 0 issues the MMAs.  An arrival without a scope is a release at CTA
scope, which orders nothing for a thread of the other CTA.
"""
import os
import re

import pytest

from tests.test_tensor_memory_rule import CSRC, kernels

KERNEL = dict(kernels(os.path.join(CSRC, "adapter_tile.cu")))["adapter_tile_kernel"]


def test_operands_written_by_threads_are_released_and_acquired_at_cluster_scope():
    # the plain remote arrival announces only what tensor memory or copies hold
    assert re.findall(r"mbar_arrive_remote\((\w+)", KERNEL) == ["leader_accempty"]
    assert re.search(r"mbar_arrive_remote_release\(leader_passed", KERNEL)
    take = KERNEL.index("mbar_acquire_cluster(&passed[s]")
    assert KERNEL.index("mbar_arrive(&full[s])", take) > take
    with open(os.path.join(CSRC, "tcgen05.cuh")) as f:
        text = f.read()
    assert "mbarrier.arrive.release.cluster.shared::cluster.b64" in text
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in text


ALIGNED = r"\b(tmem_ld\d+\(|tmem_dealloc\w*\(|expand_token\()"
WHOLE = r"\b(__syncwarp\(|__syncthreads\(|__all_sync\([^;{]*|__any_sync\(|cluster_sync_all\()"
APART = r"\bmbar_drain\(|\bmbar_wait\(|\bif \((?!warp\b|constexpr|w \+ 2|threadIdx.x == 64 && ok|slots? >=? 0\)|r < ranks\))"


@pytest.mark.parametrize("name", ["adapter_tile_kernel", "adapter_split_kernel",
                                  "adapter_shrink_tile_kernel"])
def test_warps_are_whole_before_instructions_that_take_whole_warps(name):
    """tcgen05.ld, tcgen05.dealloc, barrier.cluster and mma.sync are .aligned: between a
    wait or a branch that lanes can leave at different times and each of them the warp
    meets again; in a loop, after its head."""
    body = dict(kernels(os.path.join(CSRC, {
        "adapter_tile_kernel": "adapter_tile.cu", "adapter_split_kernel": "adapter.cu",
        "adapter_shrink_tile_kernel": "adapter_shrink.cu"}[name])))[name]
    found = list(re.finditer(ALIGNED, body))
    assert len(found) >= 2
    for op in found:
        before = body[:op.start()]
        whole = [m.end() for m in re.finditer(WHOLE, before)][-1]
        assert not re.search(APART, before[whole:]), before[-400:]
    with open(os.path.join(CSRC, "tcgen05.cuh")) as f:
        barrier = f.read().split("void cluster_sync_all() {")[1]
    assert barrier.split()[0] == "__syncwarp();"
    # loops over columns or tokens whose bodies lanes take differently
    for head, op in {"adapter_tile_kernel": [("for (int c0 = 0; c0 < BN", "tmem_ld32(")],
                     "adapter_shrink_tile_kernel": [("for (int c = 0; c < s.R", "tmem_ld8(")],
                     "adapter_split_kernel": []}[name]:
        loop = body[body.index(head):]
        assert re.search(WHOLE, loop[:loop.index(op)])
    if name == "adapter_split_kernel":
        loop = body[body.index("for (int j = ok ? j0 + warp"):]
        assert "__syncwarp();" in loop[loop.index("if (on)"):loop.index("j0 = j1")]
