"""What is measured of the operators around the routed experts of a decoder's
mixture-of-experts block, and their plain forms.

Three operators, each reached through the package's public entry points:

``route_logits``
    routing from logits: sigmoid or softmax scores, a balance bias that only
    ranks, expert groups, top-k, renormalised and scaled weights;
``block_norm``
    the norm after a block, its gate and residual scale, the new residual
    stream and the norm before the next block, in one pass;
``adapter_linear``
    a shared projection with the low-rank adapters of many requests.

``own`` says which side ``run`` computes: False the plain form (elementary
torch operations, rounded once at the end), True the package's kernels.
"""
import math
import random

import torch

own = False

_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_STABILISER = 1e-20


# ---------------------------------------------------------------------- cases

def listed():
    def route(name, **kw):
        c = dict(name=name, op="route", score="sigmoid", bias=True, groups=1, topk_groups=1,
                 group_score="top2", renorm=True, scale=1.0, dtype="fp32", masked=0.0)
        c.update(kw)
        return c

    def norm(name, **kw):
        c = dict(name=name, op="norm", stream="bf16", post=True, gate="none", sigmoid=False,
                 scale=1.0, pre=True)
        c.update(kw)
        return c

    def adapter(name, **kw):
        c = dict(name=name, op="adapter", scaled=True, none=0.0)
        c.update(kw)
        return c

    return [
        # one token of one request being decoded: latency of the call
        route("route one token", T=1, E=384, k=8),
        # the router of a serving batch of long prompts: 8 groups of 48 experts, 4 kept
        route("route prompts, groups", T=8192, E=384, k=8, groups=8, topk_groups=4, scale=2.5),
        # softmax router on bf16 logits, ragged token count, experts taken out of service
        route("route softmax, bf16", T=2051, E=200, k=6, score="softmax", bias=False, groups=4,
              topk_groups=2, group_score="max", dtype="bf16", renorm=False, masked=0.03),
        # decode batch of 32 requests, between two blocks of a decoder of width 7168
        norm("norm decode", T=32, N=7168),
        # long prompts, gated block output, bf16 residual stream
        norm("norm prompts, gate", T=8192, N=7168, gate="full", sigmoid=True, scale=0.5),
        # fp32 residual stream of the latent width, gate per channel, odd token count
        norm("norm fp32 stream", T=2049, N=3584, stream="fp32", gate="channel"),
        # a width that no vector of 16 bytes divides: plain pre-norm of an odd head
        norm("norm odd width", T=777, N=1023, post=False, gate="token"),
        # one token with its adapter through the latent down-projection
        adapter("adapters one token", T=1, K=7168, N=3584, R=16, adapters=8, run=1),
        # 32 requests decoded together, each with its own adapter, latent up-projection
        adapter("adapters decode", T=32, K=3584, N=7168, R=16, adapters=64, run=1),
        # a larger decode batch with mixed adapters, one request in eight without one
        adapter("adapters batch", T=256, K=7168, N=2048, R=32, adapters=48, run=1, none=0.125),
        # a few prompts of about 300 tokens each, ragged
        adapter("adapters prompts", T=2047, K=7168, N=3584, R=16, adapters=16, run=300, none=0.1),
        # a full prefill batch of long prompts
        adapter("adapters prefill", T=8192, K=3584, N=7168, R=64, adapters=8, run=2000),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm, ragged rather than a multiple of 1024."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - 1 if n % 1024 == 0 else n


def _odd(n):
    return n | 1


def draw(rng):
    """One more case: sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["route", "norm", "adapter"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 8, 512 // groups)
        topk_groups = rng.randint(1, groups)
        most = min(16, topk_groups * per)
        score = rng.choice(["sigmoid", "softmax"])
        return dict(op="route", T=_log_int(rng, 1, 8192), E=groups * per, k=rng.randint(1, most),
                    score=score, bias=rng.random() < (0.8 if score == "sigmoid" else 0.3),
                    groups=groups, topk_groups=topk_groups,
                    group_score=rng.choice(["top2", "max"]), renorm=rng.random() < 0.8,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.05]))
    if op == "norm":
        N = _log_int(rng, 64, 7168)
        if rng.random() < 0.75:
            N = 64 * _odd(N // 128 * 2)
        return dict(op="norm", T=_log_int(rng, 1, 8192), N=N, stream=rng.choice(["bf16", "fp32"]),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "full", "channel", "token"]),
                    sigmoid=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.22]),
                    pre=rng.random() < 0.8)
    T = _log_int(rng, 1, 8192)
    K, N = 32 * _odd(_log_int(rng, 8, 222)), 8 * _odd(_log_int(rng, 32, 894))
    while T * K * N > 8192 * 3584 * 7168:
        K, N = 32 * _odd(K // 64), 8 * _odd(N // 16)
    return dict(op="adapter", T=T, K=K, N=N, R=8 * rng.randint(1, 8), adapters=_log_int(rng, 1, 64),
                run=1 if T <= 512 and rng.random() < 0.7 else _log_int(rng, 50, 2000),
                scaled=rng.random() < 0.7, none=rng.choice([0.0, 0.125]))


# --------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    bf16 = torch.bfloat16
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        # x of unit variance against router rows of std 0.02 at width 7168
        z = randn(T, E, std=0.02 * math.sqrt(7168)).to(_DTYPES[case["dtype"]])
        if case["masked"]:
            out = torch.rand(T, E, generator=g, device=dev) < case["masked"]
            z = torch.where(out, torch.full_like(z, -math.inf), z)
        bias = randn(E, std=0.01) if case["bias"] else None
        return {"case": case, "logits": z, "bias": bias}
    if case["op"] == "norm":
        T, N = case["T"], case["N"]
        # a residual stream has a few channels far above the rest
        loud = 1.0 + 20.0 * (torch.rand(N, generator=g, device=dev) < 0.004).float()
        s = {"case": case, "y": randn(T, N, dtype=bf16),
             "x": (randn(T, N, std=3.0) * loud).to(_DTYPES[case["stream"]]),
             "post_gain": None, "gate": None, "pre_gain": None}
        if case["post"]:
            s["post_gain"] = (1.0 + randn(N, std=0.1)).to(bf16)
        if case["pre"]:
            s["pre_gain"] = (1.0 + randn(N, std=0.1)).to(bf16)
        if case["gate"] != "none":
            shape = {"full": (T, N), "channel": (N,), "token": (T, 1)}[case["gate"]]
            s["gate"] = randn(*shape, dtype=bf16)
        return s
    T, K, N, R, A = (case[n] for n in ("T", "K", "N", "R", "adapters"))
    # requests of about `run` tokens each, one adapter to a request
    r = random.Random(seed)
    if case["run"] == 1:
        order = list(range(A))
        r.shuffle(order)
        ids = torch.tensor([order[t % A] for t in range(T)], dtype=torch.int32)
        drop = torch.tensor([r.random() < case["none"] for _ in range(T)])
        ids[drop] = -1
    else:
        ids = torch.empty(T, dtype=torch.int32)
        t = 0
        while t < T:
            n = max(1, int(case["run"] * r.uniform(0.5, 1.5)))
            ids[t:t + n] = -1 if r.random() < case["none"] else r.randrange(A)
            t += n
    scale = None
    if case["scaled"]:
        scale = 0.5 + 1.5 * torch.rand(A, generator=g, device=dev)
    return {"case": case, "x": randn(T, K, dtype=bf16), "w": randn(N, K, std=0.02, dtype=bf16),
            "lora_a": randn(A, R, K, std=0.02, dtype=bf16),
            "lora_b": randn(A, N, R, std=0.05, dtype=bf16),
            "ids": ids.to(dev), "scale": scale}


# ----------------------------------------------------------------- plain form

def _plain_route(s):
    c = s["case"]
    E, k, G, kept = c["E"], c["k"], c["groups"], c["topk_groups"]
    z = s["logits"].double()
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    there = z > -math.inf
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        top = z.amax(dim=1, keepdim=True)
        e = torch.exp(torch.where(z == top, torch.zeros_like(z), z - top))
        e = torch.where(there, e, torch.zeros_like(e))
        score = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
    key = z if s["bias"] is None else score + s["bias"].double()
    key = torch.where(there & ~torch.isnan(key), key, torch.full_like(key, -math.inf))
    outside = torch.zeros_like(there)
    if kept < G:
        # without a bias, scores stand in for the keys in a group's sum
        part = (score if s["bias"] is None else key).masked_fill(key == -math.inf, -math.inf)
        part = part.reshape(-1, G, E // G).sort(dim=2, descending=True).values
        best = key.reshape(-1, G, E // G).amax(dim=2)
        if c["group_score"] == "top2":
            two = part[:, :, :2]
            total = torch.where(two == -math.inf, torch.zeros_like(two), two).sum(dim=2)
            best = torch.where(best == -math.inf, best, total)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        inside = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        outside = ~inside.repeat_interleave(E // G, dim=1)
    first = key.sort(dim=1, descending=True, stable=True).indices
    late = outside.gather(1, first).to(torch.int8).sort(dim=1, stable=True).indices
    idx = first.gather(1, late)[:, :k]
    w = score.gather(1, idx)
    w = torch.where(key.gather(1, idx) == -math.inf, torch.zeros_like(w), w)
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + _STABILISER)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _plain_norm(s):
    c = s["case"]
    v = s["y"].float()
    if s["post_gain"] is not None:
        v = v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * s["post_gain"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        v = v * (1.0 / (1.0 + torch.exp(-gate)) if c["sigmoid"] else gate)
    r = s["x"].float() + c["scale"] * v
    h = None
    if s["pre_gain"] is not None:
        h = r * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + 1e-6) * s["pre_gain"].float()
        h = h.to(torch.bfloat16)
    return {"x": r.to(s["x"].dtype), "h": h}


def _plain_adapter(s):
    """Every row through all adapters, and all but its own set to zero."""
    x, w, A, B = s["x"].float(), s["w"].float(), s["lora_a"].float(), s["lora_b"].float()
    n, R, K = A.shape
    t = torch.matmul(x, A.reshape(n * R, K).t()).reshape(-1, n, R)
    if s["scale"] is not None:
        t = t * s["scale"].reshape(1, n, 1)
    its = s["ids"].unsqueeze(1) == torch.arange(n, device=x.device).unsqueeze(0)
    t = torch.where(its.unsqueeze(2), t, torch.zeros_like(t)).reshape(-1, n * R)
    low = torch.matmul(t, B.permute(0, 2, 1).reshape(n * R, -1))
    return (torch.matmul(x, w.t()) + low).to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        return {"route": _plain_route, "norm": _plain_norm, "adapter": _plain_adapter}[c["op"]](state)
    import int4_routed_expert_fp32_gb300 as moe
    if c["op"] == "route":
        return moe.route_logits(state["logits"], c["k"], bias=state["bias"], score=c["score"],
                                groups=c["groups"], topk_groups=c["topk_groups"],
                                group_score=c["group_score"], renorm=c["renorm"],
                                scale=c["scale"])
    if c["op"] == "norm":
        x, h = moe.block_norm(state["y"], state["x"], post_gain=state["post_gain"],
                              gate=state["gate"], gate_sigmoid=c["sigmoid"], scale=c["scale"],
                              pre_gain=state["pre_gain"], eps=1e-6)
        return {"x": x, "h": h}
    return moe.adapter_linear(state["x"], state["w"], state["lora_a"], state["lora_b"],
                              state["ids"], scale=state["scale"])


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k,
                "flops": 10 * T * E}
    if case["op"] == "norm":
        T, N = case["T"], case["N"]
        wide = 4 if case["stream"] == "fp32" else 2
        gate = {"none": 0, "full": T * N, "channel": N, "token": T}[case["gate"]]
        n = T * N * (2 + 2 * wide) + 2 * gate
        n += (2 * N if case["post"] else 0) + (2 * T * N + 2 * N if case["pre"] else 0)
        return {"bytes": n, "flops": 12 * T * N}
    T, K, N, R = (case[n] for n in ("T", "K", "N", "R"))
    # adapters in use: all of them, or as many as there are requests
    used = min(case["adapters"], max(1, T // case["run"]))
    with_one = T * (1.0 - case["none"])
    return {"bytes": 2 * (T * K + N * K + T * N) + 4 * T + used * 2 * R * (K + N),
            "flops": 2 * T * N * K + 2 * with_one * R * (K + N)}


# ------------------------------------------------------------- 64-bit values

def _exact_route(s):
    """The weights, row by row of the sorted scores in 64 bits."""
    c = s["case"]
    E, k = c["E"], c["k"]
    z = s["logits"].to(torch.float64).nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(z)
    else:
        p = torch.softmax(z, dim=1).nan_to_num(nan=0.0)
    c64 = z.clone() if s["bias"] is None else p + s["bias"].to(torch.float64)
    c64[z == -math.inf] = -math.inf
    if c["topk_groups"] < c["groups"]:
        G, n = c["groups"], E // c["groups"]
        if c["group_score"] == "max":
            value = c64.view(-1, G, n).max(dim=2).values
        else:
            base = (p if s["bias"] is None else c64).clone()
            base[z == -math.inf] = -math.inf
            two = base.view(-1, G, n).topk(min(2, n), dim=2).values
            value = two[..., 0] + (two[..., -1].clamp_min(-1e300).where(
                two[..., -1] > -math.inf, torch.zeros_like(two[..., -1])) if n > 1 else 0.0)
        keep = torch.zeros_like(value)
        keep.scatter_(1, torch.argsort(-value, dim=1, stable=True)[:, :c["topk_groups"]], 1.0)
        drop = keep.repeat_interleave(n, dim=1) == 0
        # below every kept expert, the unavailable ones too
        c64 = torch.where(c64 == -math.inf, torch.full_like(c64, -1e300), c64)
        c64[drop] = -math.inf
    idx = torch.argsort(-c64, dim=1, stable=True)[:, :k]
    w = p.gather(1, idx) * (z.gather(1, idx) > -math.inf)
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + _STABILISER)
    return [None, w * c["scale"]]


def _exact_norm(s):
    c = s["case"]
    v = s["y"].to(torch.float64)
    n = v.shape[1]
    if s["post_gain"] is not None:
        v = v / torch.sqrt((v * v).sum(dim=1) / n + 1e-6)[:, None] * s["post_gain"].to(v.dtype)
    if s["gate"] is not None:
        gate = s["gate"].to(torch.float64)
        v = v * (torch.sigmoid(gate) if c["sigmoid"] else gate)
    r = s["x"].to(torch.float64).add(v, alpha=c["scale"])
    h = None
    if s["pre_gain"] is not None:
        h = r / torch.sqrt((r * r).sum(dim=1) / n + 1e-6)[:, None] * s["pre_gain"].to(r.dtype)
    return {"x": r, "h": h}


def _exact_adapter(s):
    """Adapter by adapter over the rows that use it."""
    x = s["x"].to(torch.float64)
    y = x @ s["w"].to(torch.float64).T
    for a in sorted(set(s["ids"].tolist()) - {-1}):
        rows = torch.nonzero(s["ids"] == a).flatten()
        low = x[rows] @ s["lora_a"][a].to(torch.float64).T @ s["lora_b"][a].to(torch.float64).T
        if s["scale"] is not None:
            low = low * s["scale"][a].to(torch.float64)
        y[rows] += low
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "adapter": _exact_adapter}[case["op"]](s)
