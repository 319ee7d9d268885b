"""Packed 4-bit weights times a few rows, against 64-bit arithmetic.

Tolerance of an output, from the arithmetic: half a step of bf16 (2^-8 of the value); and of
each group of 32 columns, whose sum is built on 1032 + q in fp32: two MMAs, the
start value and its sum round at 2^-23 of at most 1040 times the group's absolute
activations each, so 4 of them, 2^-11 of scale times those (the rest of the fp32 chain
is far below).  Values below bf16's normal range: its step there, 2^-133.
"""
import pytest
import torch

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


def weights(N, K, g):
    packed = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, dtype=torch.int64)
    scale = (0.002 + 0.01 * torch.rand(N, K // 32, generator=g)).to(BF16)
    return packed.to(torch.int32).to(DEV), scale.to(DEV)


def q_of(packed):
    """[N, K] of the words' nibbles, column 8i + j in bits 4j .. 4j + 3."""
    w = packed.cpu().to(torch.int64) & 0xFFFFFFFF
    n = (w.unsqueeze(-1) >> (4 * torch.arange(8))) & 15
    return ((n ^ 8) - 8).reshape(packed.shape[0], -1).double()


def check(y, x, packed, scale):
    N, K = packed.shape[0], x.shape[1]
    s = scale.cpu().double()
    w = q_of(packed) * s.repeat_interleave(32, dim=1)
    v = x.cpu().double()
    want = v @ w.T
    by_group = v.abs().reshape(-1, K // 32, 32).sum(dim=2)
    tol = 2.0**-8 * want.abs() + 2.0**-11 * (by_group @ s.T) + 2.0**-133
    assert y.shape == (x.shape[0], N) and y.dtype == BF16
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 33, 160), (1, 300, 128), (4, 47, 1056),
         (5, 100, 2080), (8, 64, 256), (9, 40, 4128), (16, 130, 7168), (7, 31, 16384), (16, 20, 16384),
         (1, 5001, 32), (2, 2450, 1024), (13, 4999, 288), (1, 129, 28672 + 32),
         (2, 3, 1 << 20), (16, 2, (1 << 20) - 96), (1, 1 << 20, 32)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_products(moe, T, N, K):
    g = torch.Generator().manual_seed(T * 1000003 + N * 101 + K)
    packed, scale = weights(N, K, g)
    x = torch.randn(T, K, generator=g).to(BF16).to(DEV)
    y = moe.int4_matvec(x, packed, scale)
    check(y, x, packed, scale)
    assert torch.equal(y, moe.int4_matvec(x, packed, scale))


@pytest.mark.parametrize("T", [1, 2, 11])
def test_rows_that_lie_apart(moe, T):
    g = torch.Generator().manual_seed(T)
    packed, scale = weights(70, 544, g)
    wide = torch.randn(T, 544 + 24, generator=g).to(BF16).to(DEV)
    out = torch.full((T, 70), 7.0, dtype=BF16, device=DEV)
    got = moe.int4_matvec(wide[:, :544], packed, scale, out=out)
    assert got is out
    check(out, wide[:, :544], packed, scale)


def test_magnitudes(moe):
    """Any bf16 range, each row its own, zeros among them."""
    g = torch.Generator().manual_seed(3)
    packed, scale = weights(50, 640, g)
    x = torch.randn(6, 640, generator=g)
    x *= torch.tensor([1e-30, 1e30, 1.0, 0.0, 3e4, 2.0**-126]).reshape(6, 1)
    x[2, ::7] *= 2.0**-40
    x = x.to(BF16).to(DEV)
    check(moe.int4_matvec(x, packed, scale), x, packed, scale)


def test_values_that_are_not_finite_stay_in_their_row(moe):
    g = torch.Generator().manual_seed(4)
    packed, scale = weights(40, 256, g)
    x = torch.randn(11, 256, generator=g).to(BF16).to(DEV)
    clean = moe.int4_matvec(x, packed, scale)
    bad = x.clone()
    bad[3, 100], bad[9, 0] = float("nan"), float("inf")
    y = moe.int4_matvec(bad, packed, scale)
    keep = [t for t in range(11) if t not in (3, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[[3, 9]].float()).any()
    # a scale that is not finite stays in its output
    s = scale.clone()
    s[17, 2] = float("inf")
    y = moe.int4_matvec(x, packed, s)
    cols = [n for n in range(40) if n != 17]
    assert torch.equal(y[:, cols], clean[:, cols])


def test_extreme_words(moe):
    """All nibbles -8, and 7: the ends of the range in every position."""
    for word, q in ((-0x77777778, -8.0), (0x77777777, 7.0)):
        packed = torch.full((3, 16), word, dtype=torch.int32, device=DEV)
        scale = torch.ones(3, 4, dtype=BF16, device=DEV)
        x = torch.arange(1, 129, dtype=torch.float32).reshape(1, 128).to(BF16).to(DEV)
        y = moe.int4_matvec(x, packed, scale)
        want = (q * x.cpu().double().sum()).to(BF16)
        assert torch.equal(y.cpu(), want.reshape(1, 1).expand(1, 3))


def test_captured_and_replayed(moe):
    g = torch.Generator().manual_seed(5)
    packed, scale = weights(1000, 2048, g)
    a, b = (torch.randn(2, 2048, generator=g).to(BF16).to(DEV) for _ in range(2))
    want = [moe.int4_matvec(v, packed, scale) for v in (a, b)]
    x, out = a.clone(), torch.empty(2, 1000, dtype=BF16, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        moe.int4_matvec(x, packed, scale, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            moe.int4_matvec(x, packed, scale, out=out)
        for v, w in ((a, want[0]), (b, want[1]), (a, want[0])):
            x.copy_(v)
            graph.replay()
            st.synchronize()
            assert torch.equal(out, w)


def test_calls_that_follow_one_another(moe):
    """Each reads what the one before it wrote, quantised weights among them."""
    g = torch.Generator().manual_seed(6)
    w = (0.05 * torch.randn(512, 512, generator=g)).to(BF16).to(DEV)
    x = torch.randn(3, 512, generator=g).to(BF16).to(DEV)
    for _ in range(20):
        packed, scale = moe.quantize_int4(w)
        y = moe.int4_matvec(x, packed, scale)
        z = moe.int4_matvec(y, packed, scale)
        torch.cuda.synchronize()
        check(y, x, packed, scale)
        check(z, y, packed, scale)
        w = (w.float() * 0.97).to(BF16)


def test_agrees_with_the_grouped_linear(moe):
    g = torch.Generator().manual_seed(7)
    packed, scale = weights(256, 512, g)
    x = torch.randn(12, 512, generator=g).to(BF16).to(DEV)
    offsets = torch.tensor([0, 12], dtype=torch.int32, device=DEV)
    want = moe.int4_linear(x, None, offsets, packed[None], scale[None])
    got = moe.int4_matvec(x, packed, scale).float()
    # both within 2^-8 of the value and 2^-11 of the groups' absolute sums
    s = scale.double().cpu()
    tol = 2.0**-8 * want.cpu().double().abs() + 2.0**-10 * (
        x.cpu().double().abs().reshape(12, 16, 32).sum(dim=2) @ s.T)
    assert bool(((got - want).cpu().double().abs() <= tol).all())


def test_no_rows(moe):
    packed, scale = weights(8, 64, torch.Generator().manual_seed(8))
    n = moe.launch_count()
    y = moe.int4_matvec(torch.empty(0, 64, dtype=BF16, device=DEV), packed, scale)
    assert y.shape == (0, 8) and moe.launch_count() == n
