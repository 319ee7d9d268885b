"""GPU parity of grouped routing and of the fused block norm against 64-bit
references written out here row by row.

Tolerances.  Routing: the listed experts are equal; weights carry the rounding
of an fp32 exponential (2 steps of 2^-24), a sum, a division and the scale, and
a softmax the rounding of its denominator of fast exponentials (2^-22 and
|z - m| 2^-24 a term, weighted by e^-|z - m|, and 17 additions): 2e-6 in all.
Norm: one rounding to bf16 is at most 2^-8 of the value (fp32: 2^-24); before
it the fp32 arithmetic errs by at most 4e-6 of |x| + |scale v| (mean of squares
of up to 32768 values summed in 32 or more partial sums, root, division, four
products), and as much again in h's norm.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import inputs as oi

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    from int4_routed_expert_fp32_gb300.build import build
    build()
    import int4_routed_expert_fp32_gb300 as m
    torch.cuda.set_device(DEV)
    assert m.check_error() == 0
    yield m
    assert m.check_error() == 0


# ------------------------------------------------------------------- routing

def route_ref(z, k, bias=None, score="sigmoid", groups=1, topk_groups=None, group_score="top2",
              renorm=True, scale=1.0):
    """(idx, w) of logits z [T, E] (any float array), in Python and fp64."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    kept = groups if topk_groups is None else topk_groups
    per = E // groups
    idx = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k), dtype=np.float64)
    with np.errstate(all="ignore"):
        for t in range(T):
            zt = np.where(np.isnan(z[t]), -INF, z[t])
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-zt))
            else:
                top = zt.max()
                e = np.where(zt == top, 1.0, np.exp(zt - top))
                e[zt == -INF] = 0.0
                s = e / e.sum() if e.sum() > 0 else e
            key = zt.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
            key[(zt == -INF) | np.isnan(key)] = -INF
            inside = np.ones(E, dtype=bool)
            if kept < groups:
                value = []
                for g in range(groups):
                    own = range(g * per, (g + 1) * per)
                    there = sorted((key[e] for e in own if key[e] > -INF), reverse=True)
                    if not there:
                        value.append(-INF)
                    elif group_score == "max":
                        value.append(there[0])
                    elif bias is None:
                        value.append(sum(sorted((s[e] for e in own if key[e] > -INF),
                                                reverse=True)[:2]))
                    else:
                        value.append(sum(there[:2]))
                best = sorted(range(groups), key=lambda g: (-value[g], g))[:kept]
                inside = np.array([e // per in best for e in range(E)])
            order = sorted((e for e in range(E) if inside[e]), key=lambda e: (-key[e], e))[:k]
            idx[t] = order
            wt = np.array([s[e] if key[e] > -INF else 0.0 for e in order])
            w[t] = (wt / (wt.sum() + 1e-20) if renorm else wt) * scale
    return idx, w


def check_route(moe, z, k, bias=None, **kw):
    gi, gw = moe.route_logits(z, k, bias=bias, **kw)
    assert moe.check_error() == 0
    ri, rw = route_ref(z.double().cpu().numpy(), k,
                       None if bias is None else bias.double().cpu().numpy(), **kw)
    assert np.array_equal(gi.cpu().numpy(), ri)
    got = gw.double().cpu().numpy()
    assert np.all(np.abs(got - rw) <= 2e-6 * np.abs(rw) + 1e-37), np.abs(got - rw).max()


def logits(T, E, seed, std=1.7, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).to(DEV)


def ranking_bias(E, seed, std=0.01):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(E, generator=g) * std).to(DEV)


ROUTE_SHAPES = [  # T, E, k, groups, topk_groups
    (1, 384, 8, 1, 1), (33, 384, 8, 8, 4), (5, 1, 1, 1, 1), (7, 5, 3, 1, 1), (9, 8, 8, 1, 1),
    (40, 60, 4, 6, 2), (40, 200, 6, 4, 2), (12, 33, 12, 3, 2), (11, 256, 32, 8, 1),
    (6, 2048, 32, 1, 1), (4, 2048, 8, 32, 3), (5, 1088, 5, 17, 9), (600, 40, 2, 5, 5),
    (1300, 96, 6, 8, 3),
]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("shape", ROUTE_SHAPES, ids=str)
def test_route_logits(moe, shape, biased, score, dtype):
    T, E, k, groups, kept = shape
    z = logits(T, E, E + k, dtype=dtype)
    bias = ranking_bias(E, k) if biased else None
    for group_score in ("top2", "max"):
        check_route(moe, z, k, bias, score=score, groups=groups, topk_groups=kept,
                    group_score=group_score, renorm=group_score == "top2", scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,k,groups,kept", [(64, 6, 1, 1), (96, 8, 4, 2), (320, 16, 8, 3),
                                             (640, 8, 2, 1)])
def test_route_unavailable_experts(moe, E, k, groups, kept, biased, score):
    """-inf, NaN, the lowest finite value and +inf among the logits; a row
    whose mask leaves fewer than k experts, one, or none."""
    z = logits(24, E, 3)
    z[0] = -INF
    z[1] = float("nan")
    z[2] = torch.finfo(torch.float32).min
    z[3, 1:] = -INF
    z[4, :E - 2] = -INF
    z[5, ::2] = float("nan")
    z[6, 5] = INF
    z[7, 3] = INF
    z[7, E - 1] = INF
    z[8] = 0.0
    z[9] = -0.0
    z[9, ::3] = 0.0
    z[10] = 200.0
    z[11] = -200.0
    z[12, E // groups:] = -INF
    z[13] = INF
    z[14, :] = -INF
    z[14, 7] = torch.finfo(torch.float32).min
    bias = ranking_bias(E, 4) if biased else None
    if biased:
        bias[2] = -INF
        bias[9] = float("nan")
        bias[11] = 5.0
        bias[12] = -5.0
    for group_score in ("top2", "max"):
        for renorm in (True, False):
            check_route(moe, z, k, bias, score=score, groups=groups, topk_groups=kept,
                        group_score=group_score, renorm=renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_route_decides_like_64_bits(moe, score, groups, kept):
    """Keys s + b that agree to fp32 rounding: each bias is the fp32 value that
    takes its expert's key to a common target, so that the order is decided by
    what fp32 cannot see."""
    E, k = 128, 8
    z = logits(1, E, 9).repeat(40, 1)
    zz = z[0].double()
    s = torch.sigmoid(zz) if score == "sigmoid" else torch.softmax(zz, 0)
    bias = (1.0 - s).float()
    z[1:] += torch.linspace(-1e-6, 1e-6, 39, device=DEV).unsqueeze(1)
    check_route(moe, z.contiguous(), k, bias, score=score, groups=groups, topk_groups=kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept", [(24, 1, 1), (32, 1, 1), (64, 4, 2), (40, 5, 3)])
def test_route_unavailable_experts_beside_near_ties(moe, score, E, groups, kept):
    """Fewer than k experts left, some of them tied to fp32 rounding, the others
    out by logits of -inf or NaN beside biases of every kind, or by biases of -inf
    or NaN: those fill up the k in the order of their ids."""
    rng = np.random.default_rng(E)
    k = min(E // groups * kept, 20)
    base = logits(1, E, 21)[0]
    s = torch.sigmoid(base.double()) if score == "sigmoid" else torch.softmax(base.double(), 0)
    bias = (1.0 - s).float()
    other = torch.from_numpy(rng.permutation(E)[:E // 2])
    kinds = torch.tensor([0.0, 0.1, -0.3, 1e-30, -1e-30, -INF, float("nan"), 2.0])
    bias[other.to(DEV)] = kinds[torch.arange(E // 2) % 8].to(DEV)
    z = base.repeat(60, 1)
    for t in range(60):
        out = torch.from_numpy(rng.permutation(E)[:int(rng.integers(E // 2, E + 1))]).to(DEV)
        z[t, out] = -INF if t % 3 else float("nan")
    check_route(moe, z.contiguous(), k, bias, score=score, groups=groups, topk_groups=kept)


def test_route_large_logits_and_biases(moe):
    z = logits(64, 160, 5, std=40.0)
    bias = ranking_bias(160, 6, std=3.0)
    for score in ("sigmoid", "softmax"):
        check_route(moe, z, 7, bias, score=score, groups=5, topk_groups=2)
        check_route(moe, z, 7, None, score=score, groups=5, topk_groups=2)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("first,E,wide", [(0, 64, 96), (4, 64, 96), (1, 64, 96), (3, 61, 67)])
def test_route_rows_that_lie_apart(moe, dtype, first, E, wide):
    z = logits(19, wide, 12, dtype=dtype)[:, first:first + E]
    check_route(moe, z, 5, ranking_bias(E, 1), groups=1)


def test_route_no_tokens_and_defaults(moe):
    idx, w = moe.route_logits(torch.empty(0, 16, device=DEV), 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    check_route(moe, logits(3, 16, 1), 4)


@pytest.mark.parametrize("T", [1, 32, 77, 600])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_grouped_from_hidden_states(moe, T, score):
    """From x: tokens whose 64-bit decisions all have a margin of 1e-5 over the
    fp32 logits' error list the same experts; T on each logits kernel."""
    w = wl.workload("tiny", name="grouped", T=T, H=512, E=96, k=6, seed=31)
    x = wl.gen_x(w)
    W, b = wl.gen_router(w)
    kw = dict(score=score, groups=8, topk_groups=3, scale=1.5)
    terms = moe.router_prepare(W.to(DEV)) if T >= 512 else None
    gi, gw = moe.route_grouped(x.to(DEV), W.to(DEV), w.k, b.to(DEV), w_terms=terms, **kw)
    assert moe.check_error() == 0
    z = oi.x_f64(x) @ W.double().numpy().T
    ri, rw = route_ref(z, w.k, b.numpy(), **kw)
    near = np.zeros(T, dtype=bool)   # decisions that a change of 1e-5 in the logits turns
    for seed in range(6):
        shaken = z + np.random.default_rng(seed).uniform(-1e-5, 1e-5, z.shape)
        near |= (route_ref(shaken, w.k, b.numpy(), **kw)[0] != ri).any(axis=1)
    assert near.mean() < 0.2
    gi, gw = gi.cpu().numpy()[~near], gw.cpu().numpy()[~near]
    assert np.array_equal(gi, ri[~near])
    assert np.abs(gw - rw[~near]).max() <= 1e-5


def can_turn(z, idx, bias, d, score, groups, topk_groups, scale):
    """The rows of finite logits z [T, E] whose choice some change of up to d in every
    logit could turn.  A sigmoid score moves by at most d s (1 - s) (1 + d), a softmax
    score by 2 d s (1 + d); two keys can change places when they are no further apart
    than both can move, and two groups likewise with their two best."""
    T, E = z.shape
    if score == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-z))
        move = 1.01 * d * s * (1.0 - s)
    else:
        e = np.exp(z - z.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True)
        move = 2.02 * d * s
    key, shift = (z, np.full_like(z, d)) if bias is None else (s + bias, move)
    near = np.zeros(T, dtype=bool)
    for t in range(T):
        inside = np.ones(E, dtype=bool)
        if topk_groups < groups:
            per = E // groups
            best = [np.argsort(-key[t, g * per:(g + 1) * per])[:2] + g * per
                    for g in range(groups)]
            value = s[t] if bias is None else key[t]
            score_of = np.array([value[b].sum() for b in best])
            # each of the two may be another one after the change, no further off
            slack = np.array([2.0 * 1.01 * move[t, g * per:(g + 1) * per].max()
                              for g in range(groups)])
            order = np.argsort(-score_of)
            a, b = order[:topk_groups], order[topk_groups:]
            near[t] |= bool((score_of[a][:, None] - score_of[b][None] <=
                             slack[a][:, None] + slack[b][None]).any())
            inside = np.isin(np.arange(E) // per, a)
        own = np.nonzero(inside)[0]
        o = own[np.argsort(-key[t, own])][:len(idx[t]) + 1]
        near[t] |= bool((key[t, o[:-1]] - key[t, o[1:]] <= shift[t, o[:-1]] + shift[t, o[1:]]).any())
    return near


@pytest.mark.parametrize("T", [1, 31, 33, 511, 513])
@pytest.mark.parametrize("H,E,k,groups,kept,score,biased", [
    (7168, 384, 8, 8, 4, "sigmoid", True), (7168, 384, 8, 1, 1, "softmax", False),
    (1088, 200, 6, 4, 2, "softmax", True), (64, 40, 5, 5, 3, "sigmoid", False),
    (2048, 1024, 16, 1, 1, "sigmoid", True)])
def test_route_grouped_on_other_routers(moe, T, H, E, k, groups, kept, score, biased):
    """As above, on wide and narrow routers: many partial sums to a logit and one."""
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(BF16)
    W = torch.randn(E, H, generator=g) * (1.7 / H ** 0.5)
    b = torch.randn(E, generator=g) * 0.01 if biased else None
    kw = dict(score=score, groups=groups, topk_groups=kept, scale=2.5)
    gi, gw = moe.route_grouped(x.to(DEV), W.to(DEV), k, None if b is None else b.to(DEV), **kw)
    assert moe.check_error() == 0
    z = x.double().numpy() @ W.double().numpy().T
    bias = None if b is None else b.double().numpy()
    ri, rw = route_ref(z, k, bias, **kw)
    near = can_turn(z, ri, bias, 1e-5, **kw)
    assert near.mean() < 0.2
    assert np.array_equal(gi.cpu().numpy()[~near], ri[~near])
    assert np.abs(gw.cpu().numpy()[~near] - rw[~near]).max() <= 2.5e-5


# ---------------------------------------------------------------- block norm

def norm_ref(y, x, post, gate, sigmoid, scale, pre, eps):
    """(r, h, size) in fp64; size = |x| + |scale v|, what r's error goes by."""
    y = y.double().cpu()
    v = y
    if post is not None:
        v = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + eps) * post.double().cpu()
    if gate is not None:
        g = gate.double().cpu()
        v = v * (torch.sigmoid(g) if sigmoid else g)
    v = v * scale
    xx = torch.zeros_like(v) if x is None else x.double().cpu()
    r = xx + v
    inv = 1.0 / torch.sqrt((r * r).mean(dim=1, keepdim=True) + eps)
    h = None if pre is None else r * inv * pre.double().cpu()
    size = xx.abs() + v.abs()
    hsize = None if pre is None else size * inv * pre.double().cpu().abs()
    return r, h, size, hsize


def check_norm(got, ref, size, dtype, arith):
    half = torch.finfo(dtype).eps / 2
    err = (got.double().cpu() - ref).abs()
    assert torch.all(err <= half * ref.abs() * (1 + arith) + arith * size + 1e-37), \
        float((err - half * ref.abs()).max())


def norm_inputs(T, N, stream, gate, seed):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    y = randn(T, N).to(BF16).to(DEV)
    x = None if stream is None else (3 * randn(T, N)).to(stream).to(DEV)
    post, pre = ((1 + 0.1 * randn(N)).to(BF16).to(DEV) for _ in range(2))
    shape = {"none": None, "full": (T, N), "channel": (N,), "token": (T, 1)}[gate]
    return y, x, post, pre, None if shape is None else randn(*shape).to(BF16).to(DEV)


NORM_SHAPES = [(1, 7168), (3, 64), (17, 256), (9, 512), (65, 1024), (5, 1088), (400, 2048),
               (2, 8200), (1, 32768), (3, 1), (4, 7), (6, 1023), (2, 16385), (0, 64)]


@pytest.mark.parametrize("stream", [BF16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "full", "channel", "token"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_block_norm(moe, shape, gate, stream):
    T, N = shape
    y, x, post, pre, gv = norm_inputs(T, N, stream, gate, 7 * T + N)
    if gv is not None and N == 1 and gate == "token":
        pytest.skip("one column: the same tensor as a full gate")
    for use_post, use_pre, sigmoid in [(True, True, True), (False, True, False),
                                       (True, False, False)]:
        p, q = post if use_post else None, pre if use_pre else None
        gx, gh = moe.block_norm(y, x, post_gain=p, gate=gv, gate_sigmoid=sigmoid, scale=0.37,
                                pre_gain=q, eps=1e-5)
        assert moe.check_error() == 0
        assert gx.dtype == stream and (gh is None) == (q is None)
        r, h, size, hsize = norm_ref(y, x, p, gv, sigmoid, 0.37, q, 1e-5)
        check_norm(gx, r, size, stream, 4e-6)
        if q is not None:
            check_norm(gh, h, hsize, BF16, 8e-6)


@pytest.mark.parametrize("stream", [BF16, torch.float32])
@pytest.mark.parametrize("N", [3136, 6144, 7168, 8192 + 8, 16384])
def test_block_norm_wide_rows_of_many_tokens(moe, N, stream):
    """More rows than two to an SM: the variants with several vectors to a thread."""
    y, x, post, pre, gate = norm_inputs(310, N, stream, "full", N)
    gx, gh = moe.block_norm(y, x, post_gain=post, gate=gate, gate_sigmoid=True, scale=0.37,
                            pre_gain=pre, eps=1e-5)
    assert moe.check_error() == 0
    r, h, size, hsize = norm_ref(y, x, post, gate, True, 0.37, pre, 1e-5)
    check_norm(gx, r, size, stream, 4e-6)
    check_norm(gh, h, hsize, BF16, 8e-6)


def test_block_norm_without_residual_is_rmsnorm(moe):
    y, _, _, pre, _ = norm_inputs(37, 512, None, "none", 3)
    x_out, h = moe.block_norm(y, pre_gain=pre, eps=1e-6)
    assert torch.equal(x_out, y)
    assert torch.equal(h, moe.rmsnorm(y, pre, 1e-6))


@pytest.mark.parametrize("N", [384, 2048, 999])
@pytest.mark.parametrize("stream", [BF16, torch.float32])
def test_block_norm_in_place_and_strided(moe, N, stream):
    """x_out = x and h = y in place, and rows inside wider buffers: the values
    of the plain call, and nothing written between the rows."""
    T = 21
    y, x, post, pre, gate = norm_inputs(T, N, stream, "full", 5)
    kw = dict(post_gain=post, gate_sigmoid=True, pre_gain=pre, scale=0.5)
    want_x, want_h = moe.block_norm(y, x, gate=gate, **kw)
    for pad in (8, 3):
        wide = [torch.full((T, N + 2 * pad), 7.0, dtype=d, device=DEV)
                for d in (BF16, stream, BF16, stream, BF16)]
        yw, xw, gw, xo, ho = (b[:, pad:pad + N] for b in wide)
        for dst, src in ((yw, y), (xw, x), (gw, gate)):
            dst.copy_(src)
        moe.block_norm(yw, xw, gate=gw, x_out=xo, h_out=ho, **kw)
        assert torch.allclose(xo.float(), want_x.float(), rtol=2 ** -7, atol=1e-5)
        assert torch.allclose(ho.float(), want_h.float(), rtol=2 ** -7, atol=1e-5)
        for b in wide:
            assert torch.all(b[:, :pad] == 7.0) and torch.all(b[:, pad + N:] == 7.0)
    x2, y2 = x.clone(), y.clone()
    moe.block_norm(y2, x2, gate=gate, x_out=x2, h_out=y2, **kw)
    assert torch.equal(x2, want_x) and torch.equal(y2, want_h)


def test_block_norm_infinities_and_nan_stay_in_their_row(moe):
    y, x, post, pre, _ = norm_inputs(6, 640, BF16, "none", 8)
    y[1, 5] = float("nan")
    x[3, 7] = INF
    gx, gh = moe.block_norm(y, x, post_gain=post, pre_gain=pre)
    fine = [0, 2, 4, 5]
    a, b = moe.block_norm(y[fine], x[fine], post_gain=post, pre_gain=pre)
    assert torch.equal(gx[fine], a) and torch.equal(gh[fine], b)
    assert torch.isnan(gx[1]).all() and torch.isnan(gh[1]).all()
    assert gx[3, 7] == INF and torch.isnan(gh[3, 7])


# ------------------------------------------------- streams, graphs, launches

def test_ops_follow_the_current_stream_and_capture(moe):
    """The calls run on torch's current stream and replay from a graph."""
    z, bias = logits(50, 96, 2), ranking_bias(96, 2)
    y, x, post, pre, _ = norm_inputs(50, 640, BF16, "none", 4)
    want = (*moe.route_logits(z, 6, bias, groups=8, topk_groups=3),
            *moe.block_norm(y, x, post_gain=post, pre_gain=pre))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n0 = moe.launch_count()
    with torch.cuda.stream(side):
        got = (*moe.route_logits(z, 6, bias, groups=8, topk_groups=3),
               *moe.block_norm(y, x, post_gain=post, pre_gain=pre))
    assert moe.launch_count() - n0 == 2
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    zin, yin = torch.zeros_like(z), torch.zeros_like(y)
    with torch.cuda.graph(graph):
        outs = (*moe.route_logits(zin, 6, bias, groups=8, topk_groups=3),
                *moe.block_norm(yin, x, post_gain=post, pre_gain=pre))
    zin.copy_(z)
    yin.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert moe.check_error() == 0


@pytest.mark.parametrize("stream", [BF16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "full", "channel", "token"])
@pytest.mark.parametrize("T,N", [(700, 65), (900, 129), (333, 2049), (1300, 4099), (400, 7001),
                                 (310, 9003), (23, 16383), (640, 71), (5, 12345)])
def test_block_norm_odd_widths_over_many_rows(moe, T, N, gate, stream):
    """Dense rows whose 16-byte boundaries move from row to row, several rows to
    a CTA: x_out and h, x_out alone, and the pre-norm alone."""
    y, x, post, pre, gv = norm_inputs(T, N, stream, gate, T + N)
    for use_post, use_pre, sigmoid in [(True, True, True), (False, True, False),
                                       (True, False, False), (False, False, True)]:
        p, q = post if use_post else None, pre if use_pre else None
        gx, gh = moe.block_norm(y, x, post_gain=p, gate=gv, gate_sigmoid=sigmoid, scale=1.3,
                                pre_gain=q, eps=1e-6)
        r, h, size, hsize = norm_ref(y, x, p, gv, sigmoid, 1.3, q, 1e-6)
        check_norm(gx, r, size, stream, 4e-6)
        if q is not None:
            check_norm(gh, h, hsize, BF16, 8e-6)
    x2, y2 = x.clone(), y.clone()
    want = moe.block_norm(y, x, post_gain=post, gate=gv, pre_gain=pre)
    moe.block_norm(y2, x2, post_gain=post, gate=gv, pre_gain=pre, x_out=x2, h_out=y2)
    assert torch.equal(x2, want[0]) and torch.equal(y2, want[1])
    assert moe.check_error() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,k,groups,kept", [(512, 16, 8, 2), (500, 32, 4, 2), (384, 8, 8, 1),
                                             (300, 30, 1, 1), (2048, 32, 16, 2)])
def test_route_few_lanes_hold_the_kept_groups(moe, E, k, groups, kept, biased, score):
    """k near the lanes that hold the kept groups, or near 32; equal logits."""
    z = logits(60, E, E + k)
    z[40:50] = z[40:50].round(decimals=1)
    z[50:] = 0.5
    z[55:, ::7] = 1.5
    for group_score in ("top2", "max"):
        check_route(moe, z, k, ranking_bias(E, 3) if biased else None, score=score,
                    groups=groups, topk_groups=kept, group_score=group_score)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("E,k,groups,kept", [(64, 4, 8, 3), (384, 8, 8, 4), (700, 6, 7, 2)])
def test_route_groups_of_scores_below_fp32(moe, E, k, groups, kept, dtype):
    """Sigmoid scores that all are below the smallest normal fp32 value: the
    groups' order is still that of their 64-bit sums."""
    for top in (-80.0, -89.0, -105.0, -200.0):
        z = top - logits(12, E, E + k).abs().to(dtype) * 4
        check_route(moe, z.to(dtype).contiguous(), k, groups=groups, topk_groups=kept)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("E,groups,kept,ties,target", [(384, 1, 1, 12, 2.0), (96, 1, 1, 30, 0.5),
                                                       (200, 4, 4, 9, -3.0), (256, 8, 3, 16, 1.5),
                                                       (640, 1, 1, 20, 40.0)])
def test_route_near_ties_among_few(moe, E, groups, kept, ties, target, dtype, score):
    """A few experts whose keys s + b agree to fp32's rounding, far above the
    others: their order, different in every row, is that of 64 bits."""
    T, k = 300, 8
    z = logits(T, E, E + ties)
    at = torch.randperm(E, generator=torch.Generator().manual_seed(ties))[:ties].to(DEV)
    z[:, at] = logits(1, ties, 5)
    z[:, at] *= 1 + torch.linspace(-1, 1, T, device=DEV).unsqueeze(1) * 2e-6
    z = z.to(dtype)
    zz = z[T // 2].double()
    s = torch.sigmoid(zz) if score == "sigmoid" else torch.softmax(zz, 0)
    bias = ranking_bias(E, 1) + (target - 6.0)
    bias[at] = (target - s[at]).float()
    check_route(moe, z.contiguous(), k, bias, score=score, groups=groups, topk_groups=kept)
