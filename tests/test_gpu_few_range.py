"""Small values in the operators of a few tokens: h goes as the square of x, and neither it
nor the latent input u may be lost below fp16's range.

Tolerance, as relative L2 of each token's output: that of the ordinary sizes
(tests/test_gpu_few.py), and for 16 columns of h that are stored as they are, the largest
of them 2^-11 or more, fp16's step below its normal range: 2^-25 in each, 2^-23 together,
2^-12 of them.  Latent layers have the same for u.
"""
import math

import pytest
import torch

from tests.test_gpu_few import BF16, DEV, TOL, dense, experts, layer64, layer_weights, moe, routed, routing

pytestmark = pytest.mark.gpu
POWERS = [0, -6, -8, -10, -12, -16, -20, -30, -45]


def close(got, want, tol):
    e = (got.double() - want).norm(dim=1)
    n = want.norm(dim=1)
    assert bool((n > 0).all())
    assert bool((e <= tol * n).all()), (e / n).tolist()


def tokens(g, T, width):
    by = torch.tensor([2.0**POWERS[t % len(POWERS)] for t in range(T)]).reshape(T, 1)
    return (torch.randn(T, width, generator=g) * by).to(BF16).to(DEV)


@pytest.mark.parametrize("T,D,E,k,I", [(9, 256, 6, 3, 128), (9, 320, 8, 3, 192), (18, 128, 4, 2, 2112),
                                       (1, 64, 1, 1, 64), (30, 2304, 7, 4, 320), (9, 256, 6, 3, 256),
                                       (32, 64, 64, 32, 64)])
def test_experts_of_small_tokens(moe, T, D, E, k, I):
    g = torch.Generator().manual_seed(T + D + I)
    w = experts(g, E, D, I)
    idx, p = routing(g, T, E, k)
    x = tokens(g, T, D) if T > 1 else (2.0**-12 * torch.randn(1, D, generator=g)).to(BF16).to(DEV)
    y = moe.experts_few(idx, p, x, w)
    close(y, routed(w, idx, p, x.double()), TOL + 2.0**-12)
    assert torch.equal(y, moe.experts_few(idx, p, x, w))
    # an ordinary token has the same bits whatever the sizes of those beside it
    ordinary = [t for t in range(T) if POWERS[t % len(POWERS)] == 0 and T > 1]
    other = torch.randn(T, D, generator=g).to(BF16).to(DEV)
    other[ordinary] = x[ordinary]
    assert torch.equal(moe.experts_few(idx, p, other, w)[ordinary], y[ordinary])


def test_experts_with_small_weights(moe):
    g = torch.Generator().manual_seed(1)
    w = experts(g, 5, 256, 192)
    for e in range(5):
        w["up_scale"][e] *= 2.0**(-6 * e)
    idx, p = routing(g, 7, 5, 1)
    x = torch.randn(7, 256, generator=g).to(BF16).to(DEV)
    close(moe.experts_few(idx, p, x, w), routed(w, idx, p, x.double()), TOL + 2.0**-12)


@pytest.mark.parametrize("col", [0, 16, 64, 80, 176])
def test_sixteen_small_columns_that_alone_count(moe, col):
    """The other half of their group of 32 is of ordinary size, and has weights of zero.

    Its products are sums of 1032 h and 72 h that cancel against their start value: the
    start's own sum, its addition and eight MMAs round at 2^-23 of at most 1040 times the
    group's absolute h each, in all 10 * 1040 * 2^-23 < 2^-9 of scale times those.  A
    small half that was taken by the other half's unit would be off by 2^20 and more."""
    g = torch.Generator().manual_seed(2)
    w = experts(g, 2, 128, 192)
    w["up_scale"][:, col:col + 16] *= 2.0**-20
    w["down_scale"][:, :, [i for i in range(6) if i != col // 32]] = 0.0
    w["down_packed"][:, :, (col ^ 16) // 8:(col ^ 16) // 8 + 2] = 0
    idx, p = routing(g, 4, 2, 1)
    x = torch.randn(4, 128, generator=g).to(BF16).to(DEV)
    want = routed(w, idx, p, x.double())
    tol = (TOL + 2.0**-12) * want.norm(dim=1, keepdim=True) / math.sqrt(128)
    by_group = torch.empty_like(want)
    for t in range(4):
        e, v = int(idx[t, 0]), x[t].double()
        a = dense(w["gate_packed"][e], w["gate_scale"][e]) @ v
        h = a / (1 + torch.exp(-a)) * (dense(w["up_packed"][e], w["up_scale"][e]) @ v)
        sums = h.abs().reshape(6, 32).sum(dim=1)
        by_group[t] = p[t, 0].double() * (w["down_scale"][e].double() @ sums)
    off = moe.experts_few(idx, p, x, w).double() - want
    assert bool((off.norm(dim=1) <= (tol + 2.0**-9 * by_group).norm(dim=1)).all())


def test_padded_rows_beside_small_ones(moe):
    g = torch.Generator().manual_seed(3)
    w = experts(g, 3, 192, 64)
    idx, p = routing(g, 8, 3, 2)
    x = tokens(g, 8, 192)
    x[[1, 5]] = 0.0
    y = moe.experts_few(idx, p, x, w)
    keep = [0, 2, 3, 4, 6, 7]
    close(y[keep], routed(w, idx, p, x.double())[keep], TOL + 2.0**-12)
    assert not y[[1, 5]].any()


LAYERS = [dict(T=9, H=256, E=6, k=2, I=128), dict(T=9, H=320, E=6, k=2, I=192, L=576, norm=True),
          dict(T=9, H=320, E=6, k=2, I=192, L=576), dict(T=18, H=128, E=5, k=3, I=64, L=2112, norm=True),
          dict(T=9, H=256, E=6, k=2, I=256, L=512, norm=True), dict(T=9, H=192, E=4, k=2, I=64, S=128),
          dict(T=20, H=192, E=7, k=2, I=64, L=320, S=128)]


@pytest.mark.parametrize("c", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_layers_of_small_tokens(moe, c):
    g = torch.Generator().manual_seed(sum(c.values()))
    w = layer_weights(g, c["H"], c["E"], c["I"], c.get("L", 0), c.get("S", 0), c.get("norm", False))
    x = tokens(g, c["T"], c["H"])
    y = moe.layer_few(x, w, c["k"])
    close(y, layer64(w, x, c["k"]), TOL + 2.0**-11)
    assert torch.equal(y, moe.layer_few(x, w, c["k"]))


def test_a_norm_without_eps_gives_small_tokens_their_full_size(moe):
    g = torch.Generator().manual_seed(5)
    w = layer_weights(g, 256, 4, 128, L=128, norm=True)
    x = tokens(g, 7, 256)  # down to 2^-20: the squares of y stay in fp32's range
    y = moe.layer_few(x, w, 2, eps=0.0)
    want = layer64(w, x, 2, eps=0.0)
    close(y, want, TOL + 2.0**-11)
    assert float(want.norm(dim=1).min()) > 1.0


def test_small_tokens_captured_and_replayed(moe):
    """The record of what is small is made anew on every replay."""
    g = torch.Generator().manual_seed(6)
    w = layer_weights(g, 256, 6, 128, L=192, S=64)
    ins = [tokens(g, 9, 256), torch.randn(9, 256, generator=g).to(BF16).to(DEV), tokens(g, 9, 256)]
    want = [moe.layer_few(v, w, 2) for v in ins]
    x = ins[0].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = moe.layer_few(x, w, 2)
        for i in (0, 1, 2, 1, 0):
            x.copy_(ins[i])
            graph.replay()
            st.synchronize()
            assert torch.equal(out, want[i])
