"""Shared memory that one CTA writes and the other CTA's MMAs read is handed over at
cluster scope (no GPU needed: what is looked at is the source).

In the pair kernel of the adapter projection the low-rank operands are plain writes of
both CTAs and rank 0 issues the MMAs.  An arrival without a scope is a release at CTA
scope, which orders nothing for a thread of the other CTA.
"""
import os
import re

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
