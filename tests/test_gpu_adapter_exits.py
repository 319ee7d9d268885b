"""Exit paths of the adapter projection's kernels: copies that never arrive.

Builds of the kernels whose producers stop (as if the copies never came) run with
waits of 20 ms: the call records MOE_ERR_TIMEOUT, the context stays usable, and the
next ordinary call has the bits it had before.  Nothing faults or hangs: every wait
has its limit.
"""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
LIMIT = 20_000_000  # ns


@pytest.fixture(scope="module")
def moe():
    from int4_routed_expert_fp32_gb300.build import build
    build()
    import int4_routed_expert_fp32_gb300 as m
    torch.cuda.set_device(DEV)
    assert m.check_error() == 0
    yield m
    assert m.check_error() == 0


def inputs(T, K, N, R, n):
    g = torch.Generator().manual_seed(T + R)

    def randn(*shape, std):
        return (std * torch.randn(*shape, generator=g)).to(BF16).to(DEV)

    ids = (torch.arange(T) % n).to(torch.int32).to(DEV)
    return (randn(T, K, std=1.0), randn(N, K, std=0.02), randn(n, R, K, std=0.02),
            randn(n, N, R, std=0.1), ids)


def check(moe, args, kernel, stage):
    want = moe.adapter_linear(*args)
    assert moe.check_error() == 0
    t0 = time.monotonic()
    moe.adapter_linear_stall_selftest(*args, kernel, stage, LIMIT)
    assert moe.check_error() == moe.capi.MOE_ERR_TIMEOUT
    # a wait, and the exit's waits for what was issued: some tenths of a second
    assert time.monotonic() - t0 < 5.0
    assert moe.check_error() == 0
    for _ in range(2):
        assert torch.equal(moe.adapter_linear(*args), want)
    assert moe.check_error() == 0


@pytest.mark.parametrize("stage", [0, 1])
@pytest.mark.parametrize("T,R", [(9, 16), (64, 64), (200, 48), (300, 32), (300, 128)])
def test_low_rank_vectors_whose_copies_stop(moe, T, R, stage):
    check(moe, inputs(T, 2048, 264, R, 5), 0, stage)


@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("T,R", [(1, 16), (8, 8), (9, 16), (64, 64), (200, 48)])
def test_split_projection_whose_copies_stop(moe, T, R, stage):
    check(moe, inputs(T, 2048, 264, R, 5), 1, stage)


@pytest.mark.parametrize("T,R,n", [(1, 16, 1), (8, 8, 5), (64, 64, 60), (200, 128, 150)])
def test_split_projection_whose_low_rank_rows_never_come(moe, T, R, n):
    check(moe, inputs(T, 512, 264, R, n), 2, 0)


# K = 2048 is 32 stages; after them come those of the adapters that the tile's rows use
@pytest.mark.parametrize("stage", [0, 3, 31, 32, 33, 36])
@pytest.mark.parametrize("T,N,R", [(300, 264, 16), (600, 520, 128), (4100, 4104, 16)])
def test_tile_projection_whose_copies_stop(moe, T, N, R, stage):
    check(moe, inputs(T, 2048, N, R, 5), 1, stage)
