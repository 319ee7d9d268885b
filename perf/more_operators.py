"""What is measured of the products of 4-bit weights for a few tokens, and their
plain forms.

Three operators, each reached through the package's public entry points:

``int4_matvec``
    y = x W^T for packed int4 weights with a bf16 scale per 32 columns;
``experts_few``
    the routed experts of a few tokens whose routing is given: gate, up, SiLU,
    down and the weighted sum;
``layer_few``
    a whole mixture-of-experts layer for a few tokens: router, experts and sum,
    with the latent projections and the shared expert where the layer has them.

``own`` says which side ``run`` computes: False the plain form (elementary
torch operations, rounded once at the end), True the package's kernels.
"""
import math
import random

import torch

own = False

_GROUP = 32
_EPS = 1e-6
_MOST = 384 * 3 * 7168 * 2048  # weights of the largest listed layer's experts


# ---------------------------------------------------------------------- cases

def listed():
    def matvec(name, **kw):
        return dict(dict(name=name, op="matvec", apart=0), **kw)

    def experts(name, **kw):
        return dict(dict(name=name, op="experts"), **kw)

    def layer(name, **kw):
        return dict(dict(name=name, op="layer", L=0, norm=False, shared=0, renorm=True), **kw)

    return [
        # a narrow projection of one token: latency of the call
        matvec("matvec small", T=1, N=1024, K=2048),
        # one token through a square projection of a decoder of width 7168
        matvec("matvec one token", T=1, N=7168, K=7168),
        # three drafted tokens, an odd row count, K of 65 groups, x a slice of wider rows
        matvec("matvec drafts, odd", T=3, N=3585, K=2080, apart=96),
        # a small decode batch through a wide fused projection
        matvec("matvec batch, wide", T=16, N=16384, K=7168),
        # the experts of one token, routed elsewhere (groups, softmax)
        experts("experts one token", T=1, D=7168, E=64, k=8, I=2048, pool=64),
        # six drafted tokens on the latent width, sharing some of their experts
        experts("experts drafts", T=6, D=3584, E=384, k=8, I=1024, pool=24),
        # a small model's decode batch: widths that 256 does not divide, every expert busy
        experts("experts small model", T=29, D=576, E=48, k=5, I=320, pool=48),
        # the smallest layer of the test suite: every expert gets several of 16 tokens
        layer("layer tiny", T=16, H=256, E=8, k=2, I=128),
        # one token of one request: the latency of a decode step's layer
        layer("layer one token", T=1, H=7168, E=384, k=8, I=2048),
        # a handful of requests, an always-active shared expert, I of 44 groups
        layer("layer shared", T=5, H=4096, E=128, k=6, I=1408, shared=2816),
        # eight requests on a latent layer with its norm
        layer("layer latent", T=8, H=7168, E=384, k=8, I=1024, L=3584, norm=True),
        # a decode batch of 32 requests at full width
        layer("layer decode", T=32, H=7168, E=384, k=8, I=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi, step):
    """A multiple of ``step``, often an odd one."""
    n = max(1, _log_int(rng, lo, hi) // step)
    return step * (n | 1 if rng.random() < 0.6 else n)


def draw(rng):
    """One more case: sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["matvec", "experts", "layer"])
    if op == "matvec":
        T = _log_int(rng, 1, 16)
        K = _wide(rng, 64, 16384, 32)
        N = _log_int(rng, 16, min(32768, 16384 * 7168 // K))
        return dict(op=op, T=T, N=N, K=K, apart=rng.choice([0, 0, 8, 128]))
    T = _log_int(rng, 1, 32)
    E = _log_int(rng, 4, 384)
    k = min(E, _log_int(rng, 1, 12))
    I = _wide(rng, 64, 2048, 64)
    D = min(_wide(rng, 128, 7168, 64), 64 * max(1, _MOST // (3 * E * I * 64)))
    if op == "experts":
        return dict(op=op, T=T, D=D, E=E, k=k, I=I, pool=rng.randint(k, E))
    L = D if rng.random() < 0.3 else 0
    H = _wide(rng, 128, 7168, 64) if L else D
    return dict(op=op, T=T, H=H, E=E, k=k, I=I, L=L, norm=bool(L) and rng.random() < 0.7,
                shared=rng.choice([0, 0, _wide(rng, 64, 2048, 64)]), renorm=rng.random() < 0.8)


# --------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    def bits(*shape):
        return torch.randint(-2**31, 2**31, shape, generator=g, device=dev, dtype=torch.int32)

    def int4(*shape):
        """Packed weights [..., N, K/8] and scales [..., N, K/32] of std near 0.02: a nibble
        is the sum of two values of 0..7, less 7, as quantised weights gather round 0."""
        lead, K = shape[:-1], shape[-1]
        n = (bits(*lead, K // 8) & 0x77777777) + (bits(*lead, K // 8) & 0x77777777)
        # plus 9 in each nibble, without carries into the next
        n = ((n & 0x77777777) + 0x11111111) ^ ((n ^ -0x66666667) & -0x77777778)
        scale = 0.003 + 0.006 * torch.rand(*lead, K // _GROUP, generator=g, device=dev)
        return n, scale.to(torch.bfloat16)

    def experts(E, D, I):
        w = {}
        for name, N, K in (("gate", I, D), ("up", I, D), ("down", D, I)):
            w[name + "_packed"], w[name + "_scale"] = int4(E, N, K)
        return w

    T = case["T"]
    if case["op"] == "matvec":
        K = case["K"]
        x = randn(T, K + case["apart"])[:, :K]
        packed, scale = int4(case["N"], K)
        return {"case": case, "x": x, "packed": packed, "scale": scale}
    E, k = case["E"], case["k"]
    if case["op"] == "experts":
        r = random.Random(seed)
        pool = r.sample(range(E), case["pool"])
        idx = torch.tensor([r.sample(pool, k) for _ in range(T)], dtype=torch.int32)
        p = torch.rand(T, k, generator=g, device=dev) + 0.1
        return {"case": case, "x": randn(T, case["D"]), "idx": idx.to(dev),
                "p": p / p.sum(dim=1, keepdim=True), "weights": experts(E, case["D"], case["I"])}
    H, L, S = case["H"], case["L"], case["shared"]
    w = experts(E, L or H, case["I"])
    f32 = torch.float32
    # logits of a std near 1.7 at any width
    w["router_w"] = randn(E, H, std=1.7 / math.sqrt(H), dtype=f32)
    w["router_bias"] = randn(E, std=0.01, dtype=f32)
    if L:
        w["lat_down"], w["lat_up"] = randn(L, H, std=1 / math.sqrt(H)), randn(H, L, std=0.02)
        if case["norm"]:
            w["lat_norm"] = (1.0 + randn(L, std=0.1, dtype=f32)).to(torch.bfloat16)
    if S:
        w["shared_gate"], w["shared_up"] = randn(S, H, std=0.02), randn(S, H, std=0.02)
        w["shared_down"] = randn(H, S, std=0.02)
    return {"case": case, "x": randn(T, H), "weights": w}


# ----------------------------------------------------------------- plain form

def _weights(packed, scale):
    """fp32 [N, K] of packed words [N, K/8] and scales [N, K/32]."""
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=packed.device)
    n = (packed.unsqueeze(-1) >> shifts) & 15
    q = ((n ^ 8) - 8).float().reshape(scale.shape[0], scale.shape[1], _GROUP)
    return (q * scale.float().unsqueeze(-1)).reshape(packed.shape[0], -1)


def _plain_matvec(s):
    return torch.matmul(s["x"].float(), _weights(s["packed"], s["scale"]).t()).to(torch.bfloat16)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_experts(u, idx, p, w):
    """fp32 [T, D]: every (token, slot) through its expert, in slot order."""
    def pick(name, e):
        return _weights(w[name + "_packed"].index_select(0, e)[0],
                        w[name + "_scale"].index_select(0, e)[0])

    rows = []
    for t in range(u.shape[0]):
        total = 0.0
        for j in range(idx.shape[1]):
            e = idx[t, j:j + 1]
            h = _silu(torch.matmul(pick("gate", e), u[t])) * torch.matmul(pick("up", e), u[t])
            total = total + p[t, j] * torch.matmul(pick("down", e), h)
        rows.append(total)
    return torch.stack(rows)


def _plain_layer(s):
    c, w, x = s["case"], s["weights"], s["x"].float()
    z = torch.matmul(x.double(), w["router_w"].double().t())
    score = 1.0 / (1.0 + torch.exp(-z))
    key = score + w["router_bias"].double()
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    p = score.gather(1, idx)
    if c["renorm"]:
        p = p / (p.sum(dim=1, keepdim=True) + 1e-20)
    u = torch.matmul(x, w["lat_down"].float().t()) if c["L"] else x
    y = _plain_experts(u, idx, p.float(), w)
    if c["L"]:
        if c["norm"]:
            y = y * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + _EPS)
            y = y * w["lat_norm"].float()
        y = torch.matmul(y, w["lat_up"].float().t())
    if c["shared"]:
        h = _silu(torch.matmul(x, w["shared_gate"].float().t()))
        h = h * torch.matmul(x, w["shared_up"].float().t())
        y = y + torch.matmul(h, w["shared_down"].float().t())
    return y.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if own:
        import int4_routed_expert_fp32_gb300 as moe
        if c["op"] == "matvec":
            return moe.int4_matvec(state["x"], state["packed"], state["scale"])
        if c["op"] == "experts":
            return moe.experts_few(state["idx"], state["p"], state["x"], state["weights"])
        return moe.layer_few(state["x"], state["weights"], c["k"], renorm=c["renorm"], eps=_EPS)
    if c["op"] == "matvec":
        return _plain_matvec(state)
    if c["op"] == "experts":
        y = _plain_experts(state["x"].float(), state["idx"], state["p"], state["weights"])
        return y.to(torch.bfloat16)
    return _plain_layer(state)


def _busy(pool, k, T):
    """Expected distinct experts of T tokens that choose k of the pool each."""
    return pool * (1.0 - (1.0 - k / pool) ** T)


def work(case):
    T = case["T"]
    if case["op"] == "matvec":
        N, K = case["N"], case["K"]
        return {"bytes": N * K / 2 + N * K / 16 + 2 * T * (N + K), "flops": 2 * T * N * K}
    E, k, I = case["E"], case["k"], case["I"]
    if case["op"] == "experts":
        D, busy = case["D"], _busy(case["pool"], k, T)
        return {"bytes": busy * 3 * D * I * (1 / 2 + 1 / 16) + 4 * T * D + 8 * T * k,
                "flops": T * k * 6 * D * I}
    H, L, S = case["H"], case["L"], case["shared"]
    D = L or H
    n = _busy(E, k, T) * 3 * D * I * (1 / 2 + 1 / 16) + 4 * E * (H + 1) + 4 * T * H
    n += 4 * L * H + 6 * S * H + (2 * L if case["norm"] else 0)
    return {"bytes": n, "flops": 2 * T * (k * 3 * D * I + E * H + 2 * L * H + 3 * S * H)}


# ------------------------------------------------------------- 64-bit values

def _weights64(packed, scale):
    """Byte by byte: the low nibble of a byte comes before its high one."""
    b = packed.contiguous().view(torch.uint8)
    low = (b << 4).view(torch.int8) >> 4
    high = b.view(torch.int8) >> 4
    q = torch.stack([low, high], dim=-1).flatten(-2).to(torch.float64)
    return q.mul_(scale.to(torch.float64).repeat_interleave(_GROUP, dim=-1))


def _exact_experts(u, idx, p, w):
    """Expert by expert over the tokens that chose it."""
    out = torch.zeros_like(u)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        v = u[t]
        gate = v @ _weights64(w["gate_packed"][e], w["gate_scale"][e]).T
        up = v @ _weights64(w["up_packed"][e], w["up_scale"][e]).T
        y = (gate * torch.sigmoid(gate) * up) @ _weights64(w["down_packed"][e],
                                                           w["down_scale"][e]).T
        out.index_add_(0, t, y * p[t, j].to(torch.float64)[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    x = s["x"].to(f64)
    if case["op"] == "matvec":
        step = max(1, 2**27 // case["K"])
        return torch.cat([x @ _weights64(s["packed"][n:n + step], s["scale"][n:n + step]).T
                          for n in range(0, case["N"], step)], dim=1)
    w = s["weights"]
    if case["op"] == "experts":
        return _exact_experts(x, s["idx"], s["p"], w)
    score = torch.sigmoid(torch.einsum("th,eh->te", x, w["router_w"].to(f64)))
    rank = torch.argsort(-(score + w["router_bias"].to(f64)), dim=1, stable=True)
    idx = rank[:, :case["k"]]
    p = torch.gather(score, 1, idx)
    if case["renorm"]:
        p = p / (p.sum(dim=1, keepdim=True) + 1e-20)
    u = x @ w["lat_down"].to(f64).T if case["L"] else x
    y = _exact_experts(u, idx, p, w)
    if case["L"]:
        if case["norm"]:
            rms = ((y * y).sum(dim=1, keepdim=True) / case["L"] + _EPS).sqrt()
            y = y / rms * w["lat_norm"].to(f64)
        y = y @ w["lat_up"].to(f64).T
    if case["shared"]:
        gate = x @ w["shared_gate"].to(f64).T
        y = y + (gate * torch.sigmoid(gate) * (x @ w["shared_up"].to(f64).T)) @ \
            w["shared_down"].to(f64).T
    return y
