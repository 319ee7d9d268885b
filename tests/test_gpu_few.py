"""The routed experts, and the whole layer, of a few tokens against 64-bit arithmetic.

Tolerance, as relative L2 of each token's output: half a step of bf16 for the output
(2^-8), half a step of fp16 for h (2^-11), and for the sums, built on 1032 + q in
fp32, 2^-11 of the groups' absolute activations in gate, up and down together: below
2^-10.  Latent layers round u (fp16) and two parts of z (2^-16) more: 2^-11.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
TOL = 2.0**-8 + 2.0**-11 + 2.0**-10 + 2.0**-11


@pytest.fixture(scope="module")
def moe():
    from int4_routed_expert_fp32_gb300.build import build
    build()
    import int4_routed_expert_fp32_gb300 as m
    torch.cuda.set_device(DEV)
    assert m.check_error() == 0
    yield m
    assert m.check_error() == 0


def int4(g, E, N, K):
    packed = torch.randint(-2**31, 2**31, (E, N, K // 8), generator=g, dtype=torch.int64)
    scale = (0.5 + torch.rand(E, N, K // 32, generator=g)) / (4.6 * math.sqrt(K))
    return packed.to(torch.int32).to(DEV), scale.to(BF16).to(DEV)


def experts(g, E, D, I):
    w = {}
    for name, N, K in (("gate", I, D), ("up", I, D), ("down", D, I)):
        w[name + "_packed"], w[name + "_scale"] = int4(g, E, N, K)
    return w


def dense(packed, scale):
    w = packed.to(torch.int64) & 0xFFFFFFFF
    n = (w.unsqueeze(-1) >> (4 * torch.arange(8, device=w.device))) & 15
    q = ((n ^ 8) - 8).reshape(packed.shape[0], -1).double()
    return q * scale.double().repeat_interleave(32, dim=1)


def mlp(w, e, v):
    gate, up, down = (dense(w[n + "_packed"][e], w[n + "_scale"][e]) for n in ("gate", "up", "down"))
    a = v @ gate.T
    return (a / (1 + torch.exp(-a)) * (v @ up.T)) @ down.T


def routed(w, idx, p, u):
    out = torch.zeros_like(u)
    for t in range(u.shape[0]):
        for e, weight in zip(idx[t].tolist(), p[t].double().tolist()):
            if 0 <= e < w["gate_packed"].shape[0]:
                out[t] += weight * mlp(w, e, u[t:t + 1])[0]
    return out


def close(got, want):
    e = (got.double() - want).norm(dim=1)
    n = want.norm(dim=1)
    assert bool((e <= TOL * n + 1e-30).all()), (e / n).tolist()


def routing(g, T, E, k):
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    p = torch.rand(T, k, generator=g) + 0.05
    return idx.to(DEV), (p / p.sum(dim=1, keepdim=True)).to(DEV)


SIZES = [(1, 64, 1, 1, 64), (1, 128, 4, 2, 64), (2, 192, 5, 3, 320), (3, 256, 8, 8, 128),
         (4, 512, 16, 4, 256), (17, 320, 6, 4, 192), (32, 128, 40, 5, 64), (32, 64, 64, 32, 64),
         (5, 2112, 3, 2, 64), (4, 2304, 3, 2, 2112), (9, 4352, 4, 2, 128), (1, 7168, 8, 8, 2048),
         (7, 64, 2048, 3, 64), (31, 1024, 30, 7, 448)]


@pytest.mark.parametrize("T,D,E,k,I", SIZES)
def test_experts(moe, T, D, E, k, I):
    g = torch.Generator().manual_seed(T * 7919 + D * 31 + E)
    w = experts(g, E, D, I)
    idx, p = routing(g, T, E, k)
    x = torch.randn(T, D, generator=g).to(BF16).to(DEV)
    y = moe.experts_few(idx, p, x, w)
    assert y.shape == (T, D) and y.dtype == BF16
    close(y, routed(w, idx, p, x.double()))
    assert torch.equal(y, moe.experts_few(idx, p, x, w))


def test_choices_out_of_the_ordinary(moe):
    """All tokens at one expert, one expert twice in a token, weights of zero and below."""
    g = torch.Generator().manual_seed(1)
    w = experts(g, 6, 256, 128)
    x = torch.randn(32, 256, generator=g).to(BF16).to(DEV)
    p = torch.rand(32, 2, generator=g).to(DEV)
    same = torch.full((32, 2), 3, dtype=torch.int32, device=DEV)
    close(moe.experts_few(same, p, x, w), routed(w, same, p, x.double()))
    idx, p = routing(g, 32, 6, 3)
    p[4, 1], p[5] = 0.0, -p[5]
    close(moe.experts_few(idx, p, x, w), routed(w, idx, p, x.double()))


def test_ids_that_name_no_expert(moe):
    g = torch.Generator().manual_seed(2)
    w = experts(g, 5, 128, 64)
    idx, p = routing(g, 6, 5, 3)
    x = torch.randn(6, 128, generator=g).to(BF16).to(DEV)
    idx[1, 0], idx[2, 2], idx[4] = -1, 5, 2**31 - 1
    out = torch.full((6, 128), 9.0, dtype=BF16, device=DEV)
    moe.experts_few(idx, p, x, w, out=out)
    assert moe.check_error() == moe.capi.MOE_ERR_INVALID
    want = routed(w, idx, p, x.double())
    assert not out[4].any()
    keep = [0, 1, 2, 3, 5]
    close(out[keep], want[keep])
    idx[:] = -7  # no choice at all
    out.fill_(9.0)
    moe.experts_few(idx, p, x, w, out=out)
    assert moe.check_error() == moe.capi.MOE_ERR_INVALID
    assert not out.any()


def test_magnitudes_and_values_that_are_not_finite(moe):
    g = torch.Generator().manual_seed(3)
    w = experts(g, 8, 256, 128)
    idx, p = routing(g, 7, 8, 2)
    x = torch.randn(7, 256, generator=g)
    x[1] = 0.0
    x[2, 5] *= 1000.0
    x[3] *= 2.0**-20
    x = x.to(BF16).to(DEV)
    y = moe.experts_few(idx, p, x, w)
    want = routed(w, idx, p, x.double())
    assert not y[1].any()
    # h of the fourth token lies far below fp16's normal range: an absolute step of 2^-25
    keep = [0, 2, 4, 5, 6]
    close(y[keep], want[keep])
    bad = x.clone()
    bad[0, 3], bad[5, 200] = float("nan"), float("-inf")
    z = moe.experts_few(idx, p, bad, w)
    assert moe.check_error() == moe.capi.MOE_ERR_UNSUPPORTED  # such an h has no fp16 value
    assert torch.equal(z[[1, 2, 3, 4, 6]], y[[1, 2, 3, 4, 6]])
    assert not torch.isfinite(z[[0, 5]].float()).any()


def test_h_beyond_fp16_is_reported(moe):
    g = torch.Generator().manual_seed(4)
    w = experts(g, 2, 64, 64)
    idx, p = routing(g, 2, 2, 1)
    x = (1e4 * torch.randn(2, 64, generator=g)).to(BF16).to(DEV)
    moe.experts_few(idx, p, x, w)
    assert moe.check_error() == moe.capi.MOE_ERR_UNSUPPORTED


# ------------------------------------------------------------------- layers

def layer_weights(g, H, E, I, L=0, S=0, norm=False):
    w = experts(g, E, L or H, I)
    w["router_w"] = (torch.randn(E, H, generator=g) * 1.7 / math.sqrt(H)).to(DEV)
    w["router_bias"] = (0.01 * torch.randn(E, generator=g)).to(DEV)
    if L:
        w["lat_down"] = (torch.randn(L, H, generator=g) / math.sqrt(H)).to(BF16).to(DEV)
        w["lat_up"] = (torch.randn(H, L, generator=g) / math.sqrt(L)).to(BF16).to(DEV)
        if norm:
            w["lat_norm"] = (1 + 0.1 * torch.randn(L, generator=g)).to(BF16).to(DEV)
    if S:
        for n, shape in (("gate", (S, H)), ("up", (S, H)), ("down", (H, S))):
            w["shared_" + n] = (torch.randn(*shape, generator=g) / math.sqrt(shape[1])).to(BF16).to(DEV)
    return w


def layer64(w, x, k, renorm=True, eps=1e-6):
    x = x.double()
    s = 1 / (1 + torch.exp(-(x @ w["router_w"].double().T)))
    key = s + w["router_bias"].double()
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    p = s.gather(1, idx)
    if renorm:
        p = p / (p.sum(dim=1, keepdim=True) + 1e-20)
    u = x @ w["lat_down"].double().T if "lat_down" in w else x
    y = routed(w, idx, p, u)
    if "lat_up" in w:
        if "lat_norm" in w:
            y = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + eps) * w["lat_norm"].double()
        y = y @ w["lat_up"].double().T
    if "shared_gate" in w:
        a = x @ w["shared_gate"].double().T
        y = y + (a / (1 + torch.exp(-a)) * (x @ w["shared_up"].double().T)) @ w["shared_down"].double().T
    return y


LAYERS = [dict(T=1, H=64, E=4, k=2, I=64), dict(T=1, H=2048, E=64, k=8, I=256),
          dict(T=5, H=320, E=9, k=9, I=128, renorm=False), dict(T=32, H=256, E=8, k=2, I=128),
          dict(T=3, H=128, E=600, k=6, I=64), dict(T=2, H=7232, E=33, k=4, I=64),
          dict(T=4, H=512, E=16, k=4, I=128, S=192), dict(T=19, H=256, E=12, k=3, I=64, S=448),
          dict(T=1, H=512, E=8, k=2, I=64, L=128), dict(T=8, H=1024, E=8, k=3, I=192, L=576, norm=True),
          dict(T=13, H=192, E=6, k=2, I=64, L=320, norm=True, S=128),
          dict(T=32, H=576, E=5, k=2, I=320, L=64, S=64),
          dict(T=32, H=64, E=2048, k=32, I=64), dict(T=3, H=128, E=513, k=31, I=64, S=64)]


@pytest.mark.parametrize("c", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_layers(moe, c):
    g = torch.Generator().manual_seed(sum(c.values()))
    w = layer_weights(g, c["H"], c["E"], c["I"], c.get("L", 0), c.get("S", 0), c.get("norm", False))
    x = torch.randn(c["T"], c["H"], generator=g).to(BF16).to(DEV)
    renorm = c.get("renorm", True)
    y = moe.layer_few(x, w, c["k"], renorm=renorm)
    close(y, layer64(w, x, c["k"], renorm))
    assert torch.equal(y, moe.layer_few(x, w, c["k"], renorm=renorm))


def test_ties_and_near_ties_are_decided_in_64_bits(moe):
    """Equal experts (the lower id wins) and experts that differ in the last bits of their
    logits, at the border between the chosen and the others."""
    g = torch.Generator().manual_seed(11)
    H, E, k, T = 512, 24, 4, 16
    w = layer_weights(g, H, E, 64)
    base = w["router_w"].clone()
    # every third expert is a twin of the one before it, a few ulps away or equal
    for e in range(1, E, 3):
        w["router_w"][e] = base[e - 1] * (1 + 2.0**-23 * (e % 5 - 2))
        w["router_bias"][e] = w["router_bias"][e - 1]
    x = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    close(moe.layer_few(x, w, k), layer64(w, x, k))
    # no preference at all: the lowest ids
    w["router_w"].zero_()
    w["router_bias"].zero_()
    close(moe.layer_few(x, w, k), layer64(w, x, k))


def test_padded_rows_and_experts_out_of_service(moe):
    g = torch.Generator().manual_seed(12)
    w = layer_weights(g, 256, 12, 64)
    w["router_bias"][[0, 5, 7]] = -math.inf
    w["router_bias"][3] = float("nan")
    x = torch.randn(6, 256, generator=g).to(BF16).to(DEV)
    x[2:4] = 0.0
    close(moe.layer_few(x, w, 3)[[0, 1, 4, 5]], layer64(w, x, 3)[[0, 1, 4, 5]])
    assert not moe.layer_few(x, w, 3)[2:4].any()


def test_rows_that_are_not_finite_stay_by_themselves(moe):
    """NaN, infinities and values whose logits overflow, with equal experts at the border."""
    g = torch.Generator().manual_seed(15)
    w = layer_weights(g, 256, 12, 64, L=128, S=64)
    w["router_w"][5] = w["router_w"][2]
    x = torch.randn(6, 256, generator=g).to(BF16).to(DEV)
    clean = moe.layer_few(x, w, 3)
    bad = x.clone()
    bad[1, 7], bad[2, 9], bad[4] = float("nan"), float("inf"), 3e38
    y = moe.layer_few(bad, w, 3)
    assert moe.check_error() == moe.capi.MOE_ERR_UNSUPPORTED
    assert torch.equal(y[[0, 3, 5]], clean[[0, 3, 5]])
    assert not torch.isfinite(y[[1, 2, 4]].float()).all(dim=1).any()


def test_agrees_with_the_layer(moe):
    g = torch.Generator().manual_seed(13)
    w = layer_weights(g, 512, 16, 128, L=256, S=128, norm=True)
    x = torch.randn(24, 512, generator=g).to(BF16).to(DEV)
    layer = moe.MoeLayer(24, 512, 16, 4, 128, w, L=256, I_shared=128)
    a, b = layer.forward(x).double(), layer.forward_few(x).double()
    # the other path rounds u, the expert outputs' sum and the latent output to bf16
    assert float((a - b).norm() / a.norm()) <= TOL + 3 * 2.0**-8
    assert torch.equal(layer.forward_few(x[:1]), moe.layer_few(x[:1].contiguous(), w, 4))


def test_block_with_few_tokens(moe):
    g = torch.Generator().manual_seed(14)
    w = layer_weights(g, 256, 16, 128, S=64)
    gain = torch.ones(256, dtype=BF16, device=DEV)
    args = dict(k=4, groups=4, topk_groups=2, score="softmax", route_scale=1.5, next_gain=gain)
    plain, few = moe.MoeBlock(w, **args), moe.MoeBlock(w, few_tokens=True, **args)
    for T in (1, 6, 7, 40):  # 24 choices of 16 experts: the most that go this way
        x = torch.randn(T, 256, generator=g).to(DEV)
        h = moe.rmsnorm(x.to(BF16), gain, 1e-6)
        (a, ah), (b, bh) = plain.forward(x, h), few.forward(x, h)
        if T > 6:
            assert torch.equal(a, b) and torch.equal(ah, bh)
            continue
        # three roundings to bf16 on the plain path, two on the other
        assert not torch.equal(a, b)
        assert float((a - b).norm() / (a - x).norm()) <= 5 * 2.0**-8


# ------------------------------------------------------- calls in company

def test_a_decode_step_captured_and_replayed(moe):
    """Projection, layer, norm and projection as one step, other inputs each time."""
    g = torch.Generator().manual_seed(21)
    H = 512
    w = layer_weights(g, H, 16, 128, S=64)
    wp, ws = (t[0] for t in int4(g, 1, H, H))
    gain = torch.ones(H, dtype=BF16, device=DEV)
    T = 3
    x = torch.empty(T, H, dtype=BF16, device=DEV)

    def step():
        h = moe.int4_matvec(x, wp, ws)
        y = moe.layer_few(h, w, 4)
        r, n = moe.block_norm(y, h, pre_gain=gain)
        return r, moe.int4_matvec(n, wp, ws)

    inputs = [torch.randn(T, H, generator=g).to(BF16).to(DEV) for _ in range(3)]
    want = []
    for v in inputs:
        x.copy_(v)
        want.append(step())
    graphs = []
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                out = step()
            graphs.append((graph, out))
        for turn in range(4):
            for v, e in zip(inputs, want):
                for graph, out in graphs:
                    x.copy_(v)
                    graph.replay()
                    st.synchronize()
                    assert torch.equal(out[0], e[0]) and torch.equal(out[1], e[1])


def test_calls_on_two_streams_at_once(moe):
    g = torch.Generator().manual_seed(22)
    w = experts(g, 16, 1024, 512)
    idx, p = routing(g, 8, 16, 4)
    xs = [torch.randn(8, 1024, generator=g).to(BF16).to(DEV) for _ in range(2)]
    want = [moe.experts_few(idx, p, x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(moe.experts_few(idx, p, xs[i], w))
    torch.cuda.synchronize()
    assert moe.check_error() == 0
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("c", [LAYERS[1], LAYERS[7], LAYERS[9], LAYERS[10], LAYERS[12]],
                         ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_nothing_is_written_beyond_the_output_and_the_workspace(moe, c):
    """Both between guards of a fixed pattern, the workspace of exactly the stated size."""
    import ctypes
    capi = moe.capi
    g = torch.Generator().manual_seed(31)
    w = layer_weights(g, c["H"], c["E"], c["I"], c.get("L", 0), c.get("S", 0), c.get("norm", False))
    x = torch.randn(c["T"], c["H"], generator=g).to(BF16).to(DEV)
    want = moe.layer_few(x, w, c["k"])
    cfg = capi.MoeConfig(c["T"], c["H"], c["E"], c["k"], c["I"], c.get("L", 0), 16, 1, 1e-6,
                         c.get("S", 0))
    ptrs = capi.MoeWeights(*[w[n].data_ptr() if n in w else None for n in capi.WEIGHT_NAMES])
    need = capi.lib.moe_layer_few_workspace_size(ctypes.byref(cfg))
    guard, out_bytes = 65536, want.numel() * 2
    ws = torch.full((need + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((out_bytes + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    before = x.clone()
    for _ in range(2):  # the second on what the first left
        rc = capi.lib.moe_layer_few(ctypes.byref(cfg), ctypes.byref(ptrs), x.data_ptr(),
                                    out.data_ptr() + guard, ws.data_ptr() + guard, need,
                                    torch.cuda.current_stream().cuda_stream)
        assert rc == capi.MOE_OK
        torch.cuda.synchronize()
        for t, n in ((ws, need), (out, out_bytes)):
            assert bool((t[:guard] == 0xA5).all()) and bool((t[guard + n:] == 0xA5).all())
        got = out[guard:guard + out_bytes].view(BF16).reshape(want.shape)
        assert torch.equal(got, want) and torch.equal(x, before)


@pytest.mark.parametrize("stage", [0, 1, 2])
def test_copies_that_stop_end_in_a_time_out(moe, stage):
    g = torch.Generator().manual_seed(23)
    w = experts(g, 8, 2048, 1024)
    idx, p = routing(g, 4, 8, 3)
    x = torch.randn(4, 2048, generator=g).to(BF16).to(DEV)
    want = moe.experts_few(idx, p, x, w)
    moe.experts_few_stall_selftest(idx, p, x, w, stage, 20_000_000)
    assert moe.check_error() == moe.capi.MOE_ERR_TIMEOUT
    assert torch.equal(moe.experts_few(idx, p, x, w), want)
    assert moe.check_error() == 0


def test_no_tokens(moe):
    g = torch.Generator().manual_seed(24)
    w = layer_weights(g, 64, 4, 64)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    n = moe.launch_count()
    none = torch.empty(0, 2, device=DEV)
    assert moe.layer_few(x, w, 2).shape == (0, 64)
    assert moe.experts_few(none.to(torch.int32), none, x, w).shape == (0, 64)
    assert moe.launch_count() == n
