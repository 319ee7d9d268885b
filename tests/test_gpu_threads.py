"""Calls from several host threads at once, each on its own stream and with its
own sizes: every one succeeds, with the bits of the same call made alone.

The sizes differ in the shared memory that their kernels ask for, which the
runtime keeps per kernel, not per call.
"""
import threading

import pytest
import torch

import workloads as wl
from tests._helpers import device_weights

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from int4_routed_expert_fp32_gb300.build import build
    build()
    import int4_routed_expert_fp32_gb300 as m
    torch.cuda.set_device(DEV)
    assert m.check_error() == 0
    yield m
    assert m.check_error() == 0


def randn(*shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).to(BF16).to(DEV)


def together(calls, rounds):
    """Runs each call `rounds` times in a thread of its own; the errors, and the
    last outputs."""
    errors, last = [], [None] * len(calls)
    gate = threading.Barrier(len(calls))

    def work(i):
        torch.cuda.set_device(DEV)
        stream = torch.cuda.Stream()
        try:
            with torch.cuda.stream(stream):
                gate.wait()
                for n in range(rounds):
                    last[i] = calls[i]()
                    if n % 64 == 63:
                        stream.synchronize()
            stream.synchronize()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors, last


def same(got, want):
    if isinstance(want, torch.Tensor):
        return torch.equal(got, want)
    return all(torch.equal(g, w) for g, w in zip(got, want))


def check(moe, calls, rounds):
    want = [c() for c in calls]
    torch.cuda.synchronize()
    errors, last = together(calls, rounds)
    assert not errors, errors
    assert all(same(g, w) for g, w in zip(last, want))
    assert moe.check_error() == 0


@pytest.mark.parametrize("shapes", [
    # T, K, N, R, adapters: the split kernel, alone and beside the shrink
    [(3, 256, 136, 16, 2), (64, 512, 520, 64, 9), (200, 512, 264, 48, 30)],
    # the one-launch form
    [(1, 256, 136, 8, 2), (8, 2048, 520, 8, 3), (1, 512, 264, 64, 4)],
    # the tile kernel: both kernels of long calls
    [(300, 256, 136, 16, 2), (700, 512, 520, 128, 5), (40, 512, 264, 32, 6)],
], ids=str)
def test_adapter_linear_of_several_threads(moe, shapes):
    calls = []
    for i, (T, K, N, R, n) in enumerate(shapes):
        ids = (torch.arange(T) * 7 % (n + 1) - 1).to(torch.int32).to(DEV)
        args = (randn(T, K, seed=i), randn(N, K, seed=10 + i, std=0.02),
                randn(n, R, K, seed=20 + i, std=0.02), randn(n, N, R, seed=30 + i, std=0.1), ids)
        calls.append(lambda args=args: moe.adapter_linear(*args))
    check(moe, calls, 1500)


@pytest.mark.parametrize("widths", [(8193, 12001, 16381), (12501, 20011, 32767)], ids=str)
def test_block_norm_of_several_threads(moe, widths):
    """Odd widths of dense rows (gains in shared memory), and of rows that are too
    wide for that (the row in shared memory)."""
    calls = []
    for i, N in enumerate(widths):
        y, x, g = randn(3, N, seed=i), randn(3, N, seed=10 + i), randn(N, seed=20 + i)
        calls.append(lambda y=y, x=x, g=g: moe.block_norm(y, x, post_gain=g, pre_gain=g))
    check(moe, calls, 1500)


def test_latent_layers_of_several_threads(moe):
    """Latent norms too wide for 48 KiB of shared memory."""
    calls = []
    for i, L in enumerate((12544, 14080, 16384)):
        w = wl.workload("tiny", name="threads", T=2, H=64, L=L, E=4, k=2, I=64, seed=i)
        layer = moe.MoeLayer(w.T, w.H, w.E, w.k, w.I, device_weights(w, DEV), L=L)
        x = randn(w.T, w.H, seed=i)
        calls.append(lambda layer=layer, x=x: layer.forward(x))
    check(moe, calls, 600)
