"""Refusals of grouped routing, the block norm and the adapter projection: by
the Python binding on host tensors, and by the C entry points before any launch
(no GPU needed)."""
import ctypes
import types

import pytest
import torch

CUDA_ONLY = "must live on a CUDA device"
FAKE = 0x10000  # an aligned non-null address that no refused call reads


@pytest.fixture(scope="module")
def capi():
    from int4_routed_expert_fp32_gb300.build import build
    build()
    from int4_routed_expert_fp32_gb300 import capi as c
    return c


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(*shape, dtype=torch.float32)


def raises(match, fn, *args, **kwargs):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kwargs)


def test_route_logits_binding(capi):
    r = capi.route_logits
    raises(CUDA_ONLY, r, f32(4, 16), 2)
    raises(CUDA_ONLY, r, bf16(4, 16), 2, f32(16), groups=4, topk_groups=2)
    raises(CUDA_ONLY, r, f32(4, 24)[:, 3:19], 2)          # rows that lie apart
    raises("logits: expected torch.float32", r, f32(4, 16).double(), 2)
    raises("logits: expected shape", r, f32(16), 2)
    raises("logits: its rows", r, f32(16, 4).t(), 2)
    raises("logits: its rows", r, f32(1, 16).expand(4, 16), 2)
    raises("bias: expected shape", r, f32(4, 16), 2, f32(15))
    raises("bias: expected torch.float32", r, f32(4, 16), 2, bf16(16))
    raises("score: expected one of", r, f32(4, 16), 2, score="tanh")
    raises("group_score: expected one of", r, f32(4, 16), 2, group_score="mean")


def test_route_grouped_binding(capi):
    r = capi.route_grouped
    raises(CUDA_ONLY, r, bf16(4, 64), f32(16, 64), 2)
    raises("w_router: expected shape", r, bf16(4, 64), f32(16, 32), 2)
    raises("x: expected torch.bfloat16", r, f32(4, 64), f32(16, 64), 2)
    raises("w_terms: expected shape", r, bf16(4, 64), f32(16, 64), 2, w_terms=bf16(2, 16, 64))


def test_route_options_are_read_anew_on_every_call(capi, monkeypatch):
    """A scale (or another option) held in a tensor and changed in place between two
    calls: the second call uses the new value."""
    seen = []

    def fake(cfg, *rest):
        c = cfg.contents
        seen.append((c.k, c.groups, c.topk_groups, c.renorm, c.scale))
        return 0

    names = ("moe_route_logits", "moe_route_grouped")
    monkeypatch.setattr(capi, "lib", types.SimpleNamespace(
        moe_route_grouped_workspace_size=lambda *a: 256, **{n: fake for n in names}))
    monkeypatch.setattr(capi, "_device_of", lambda *a: torch.device("cpu"))
    monkeypatch.setattr(capi, "_placed", lambda **k: torch.device("cpu"))
    monkeypatch.setattr(capi, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(capi, "_stream", lambda: None)
    scale, renorm = torch.tensor(2.5), torch.tensor(True)
    k, groups, kept = torch.tensor(2), torch.tensor(4), torch.tensor(2)
    calls = (lambda: capi.route_logits(f32(4, 16), k, groups=groups, topk_groups=kept,
                                       renorm=renorm, scale=scale),
             lambda: capi.route_grouped(bf16(4, 64), f32(16, 64), k, groups=groups,
                                        topk_groups=kept, renorm=renorm, scale=scale))
    for call in calls:
        scale.fill_(2.5), renorm.fill_(True), k.fill_(2), groups.fill_(4), kept.fill_(2)
        assert call()[0].shape == (4, 2)
        scale.fill_(1.0), renorm.fill_(False), k.fill_(3), groups.fill_(8), kept.fill_(4)
        assert call()[0].shape == (4, 3)
    assert seen == 2 * [(2, 4, 2, 1, 2.5), (3, 8, 4, 0, 1.0)]
    capi.route_logits(f32(4, 16), 2, scale=2)
    assert seen[-1] == (2, 1, 1, 1, 2.0)


def route_config(capi, **kw):
    c = dict(E=16, k=2, score=0, groups=4, topk_groups=2, group_score=0, renorm=1, scale=1.0)
    c.update(kw)
    return capi.MoeRouteConfig(*c.values())


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), "INVALID"), (dict(k=0), "INVALID"), (dict(score=2), "INVALID"),
    (dict(score=-1), "INVALID"), (dict(groups=0), "INVALID"), (dict(topk_groups=0), "INVALID"),
    (dict(topk_groups=5), "INVALID"), (dict(group_score=2), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(scale=float("inf")), "INVALID"),
    (dict(groups=3), "UNSUPPORTED"), (dict(E=4096), "UNSUPPORTED"),
    (dict(E=66, groups=33), "UNSUPPORTED"), (dict(k=9), "UNSUPPORTED"),
    (dict(E=64, k=33, topk_groups=4), "UNSUPPORTED"),
])
def test_route_config_refusals(capi, kw, code):
    L, want = capi.lib, getattr(capi, "MOE_ERR_" + code)
    cfg = ctypes.byref(route_config(capi, **kw))
    n = capi.launch_count()
    assert L.moe_route_logits(cfg, FAKE, 0, 4096, None, 4, FAKE, FAKE, None) == want
    assert L.moe_route_grouped(cfg, FAKE, FAKE, None, None, 4, 64, FAKE, FAKE, FAKE, 1 << 30,
                               None) == want
    assert capi.launch_count() == n


def test_route_argument_refusals(capi):
    L, cfg = capi.lib, ctypes.byref(route_config(capi))
    bad, uns = capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED
    n = capi.launch_count()
    assert L.moe_route_logits(None, FAKE, 0, 16, None, 4, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, None, 0, 16, None, 4, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, FAKE, 0, 15, None, 4, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, FAKE, 0, 16, None, -1, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, FAKE + 2, 0, 16, None, 4, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, FAKE, 0, 16, FAKE + 1, 4, FAKE, FAKE, None) == bad
    assert L.moe_route_logits(cfg, FAKE, 0, 16, None, 4, None, FAKE, None) == bad
    assert L.moe_route_logits(cfg, None, 0, 16, None, 0, None, None, None) == capi.MOE_OK
    g = L.moe_route_grouped
    assert g(cfg, FAKE, FAKE, None, None, 4, 100, FAKE, FAKE, FAKE, 1 << 30, None) == uns
    assert g(cfg, None, FAKE, None, None, 4, 64, FAKE, FAKE, FAKE, 1 << 30, None) == bad
    assert g(cfg, FAKE, FAKE, None, None, 4, 64, FAKE, FAKE, FAKE + 16, 1 << 30, None) == bad
    assert g(cfg, FAKE, FAKE, None, None, 4, 64, FAKE, FAKE, FAKE, 16, None) == \
        capi.MOE_ERR_WORKSPACE
    assert L.moe_route_grouped_workspace_size(cfg, 4, 64) >= 4 * 16 * 4
    assert L.moe_route_grouped_workspace_size(None, 4, 64) == 0
    assert capi.launch_count() == n


def test_block_norm_binding(capi):
    f = capi.block_norm
    raises(CUDA_ONLY, f, bf16(4, 64), bf16(4, 64), pre_gain=bf16(64))
    raises(CUDA_ONLY, f, bf16(4, 64), f32(4, 64), post_gain=bf16(64), gate=bf16(4, 1))
    raises(CUDA_ONLY, f, bf16(4, 70)[:, 3:67], None, gate=bf16(64))
    raises("y: expected torch.bfloat16", f, f32(4, 64))
    raises("y: its rows", f, bf16(64, 4).t())
    raises("x: expected shape", f, bf16(4, 64), bf16(4, 65))
    raises("x: expected torch.bfloat16", f, bf16(4, 64), bf16(4, 64).half())
    raises("post_gain: expected shape", f, bf16(4, 64), post_gain=bf16(32))
    raises("pre_gain: expected torch.bfloat16", f, bf16(4, 64), pre_gain=f32(64))
    raises("gate: expected shape", f, bf16(4, 64), gate=bf16(3, 64))
    raises("gate: expected shape", f, bf16(4, 64), gate=bf16(3, 1))
    raises("gate: expected shape", f, bf16(4, 64), gate=bf16(32))
    raises("gate: its rows", f, bf16(4, 64), gate=bf16(1, 1).expand(4, 1))
    raises("x_out: expected torch.float32", f, bf16(4, 64), f32(4, 64), x_out=bf16(4, 64))
    raises("h_out needs pre_gain", f, bf16(4, 64), h_out=bf16(4, 64))
    raises("h_out: expected shape", f, bf16(4, 64), pre_gain=bf16(64), h_out=bf16(5, 64))


def norm_args(capi, **kw):
    a = capi.MoeBlockNormArgs()
    d = dict(y=FAKE, x=FAKE, x_out=FAKE, h=FAKE, pre_gain=FAKE, y_ld=64, x_ld=64, x_out_ld=64,
             h_ld=64, T=4, N=64, scale=1.0, eps=1e-6)
    d.update(kw)
    for name, v in d.items():
        setattr(a, name, v)
    return ctypes.byref(a)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "INVALID"), (dict(N=0), "INVALID"), (dict(eps=-1.0), "INVALID"),
    (dict(eps=float("nan")), "INVALID"), (dict(scale=float("inf")), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(gate_mode=4), "INVALID"),
    (dict(gate_mode=-1), "INVALID"), (dict(gate_mode=1), "INVALID"), (dict(y=None), "INVALID"),
    (dict(x_out=None, h=None, pre_gain=None), "INVALID"), (dict(pre_gain=None), "INVALID"),
    (dict(h=None), "INVALID"), (dict(y_ld=63), "INVALID"), (dict(x_ld=0), "INVALID"),
    (dict(x_out_ld=63), "INVALID"), (dict(h_ld=63), "INVALID"),
    (dict(gate=FAKE, gate_mode=1, gate_ld=63), "INVALID"),
    (dict(gate=FAKE, gate_mode=3, gate_ld=0), "INVALID"), (dict(y=FAKE + 1), "INVALID"),
    (dict(x=FAKE + 2, x_f32=1), "INVALID"),
    (dict(N=32769, y_ld=40000, x_ld=40000, x_out_ld=40000, h_ld=40000), "UNSUPPORTED"),
])
def test_block_norm_refusals(capi, kw, code):
    n = capi.launch_count()
    assert capi.lib.moe_block_norm(norm_args(capi, **kw), None) == \
        getattr(capi, "MOE_ERR_" + code)
    assert capi.lib.moe_block_norm(None, None) == capi.MOE_ERR_INVALID
    assert capi.lib.moe_block_norm(norm_args(capi, T=0, y=None), None) == capi.MOE_OK
    assert capi.launch_count() == n


def test_struct_layouts_match_header(capi):
    from tests.test_abi import _header_struct_fields
    assert [n for n, _ in capi.MoeRouteConfig._fields_] == _header_struct_fields("moe_route_config")
    assert ctypes.sizeof(capi.MoeRouteConfig) == 8 * 4
    assert ctypes.sizeof(capi.MoeBlockNormArgs) == 12 * 8 + 7 * 4 + 4   # padded to 8 bytes


def test_adapter_linear_binding(capi):
    f = capi.adapter_linear
    T, K, N, R, n = 4, 64, 24, 8, 3

    def call(x=bf16(T, K), w=bf16(N, K), a=bf16(n, R, K), b=bf16(n, N, R),
             ids=torch.zeros(T, dtype=torch.int32), **kw):
        return f(x, w, a, b, ids, **kw)

    raises(CUDA_ONLY, call)
    raises(CUDA_ONLY, call, scale=f32(n), out=bf16(T, N))
    raises("x: expected torch.bfloat16", call, x=f32(T, K))
    raises("w: expected shape", call, w=bf16(N, K + 32))
    raises("lora_a: expected shape", call, a=bf16(n, R, K + 32))
    raises("lora_b: expected shape", call, b=bf16(n, R, N))
    raises("lora_b: expected shape", call, b=bf16(n + 1, N, R))
    raises("ids: expected torch.int32", call, ids=torch.zeros(T, dtype=torch.int64))
    raises("ids: expected shape", call, ids=torch.zeros(T + 1, dtype=torch.int32))
    raises("scale: expected shape", call, scale=f32(n + 1))
    raises("out: expected shape", call, out=bf16(T, N + 8))
    raises("x must be contiguous", call, x=bf16(K, T).t())


def test_adapter_linear_refusals(capi):
    L, n = capi.lib, capi.launch_count()
    bad, uns = capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED

    def call(T=9, K=64, N=24, R=8, adapters=3, ws_bytes=1 << 30, **ptr):
        p = dict(x=FAKE, w=FAKE, a=FAKE, b=FAKE, ids=FAKE, scale=None, y=FAKE, ws=FAKE)
        p.update(ptr)
        return L.moe_adapter_linear(p["x"], p["w"], p["a"], p["b"], p["ids"], p["scale"], T, K, N,
                                    R, adapters, p["y"], p["ws"], ws_bytes, None)

    for kw in (dict(T=-1), dict(K=0), dict(N=0), dict(R=0), dict(adapters=0), dict(x=None),
               dict(w=None), dict(a=None), dict(b=None), dict(ids=None), dict(y=None),
               dict(ws=None), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(a=FAKE + 8),
               dict(b=FAKE + 8), dict(ids=FAKE + 2), dict(scale=FAKE + 2), dict(y=FAKE + 8),
               dict(ws=FAKE + 16)):
        assert call(**kw) == bad, kw
    for kw in (dict(K=48), dict(N=20), dict(R=12), dict(R=136)):
        assert call(**kw) == uns, kw
    assert call(ws_bytes=0) == capi.MOE_ERR_WORKSPACE
    assert call(T=0, x=None) == capi.MOE_OK
    assert L.moe_adapter_linear_workspace_size(9, 64, 24, 8) >= 9 * 8 * 4
    assert L.moe_adapter_linear_workspace_size(1, 64, 24, 16) == 0   # one launch, no scratch
    assert L.moe_adapter_linear_workspace_size(0, 64, 24, 8) == 0
    assert capi.launch_count() == n


def test_moe_block_checks_its_weights(capi, monkeypatch):
    from int4_routed_expert_fp32_gb300.block import MoeBlock
    monkeypatch.setattr(capi, "router_prepare", lambda w: None)
    w = {n: None for n in capi.EXPERT_NAMES}
    w["router_w"] = f32(16, 64)
    MoeBlock(w, 2)
    raises("lat_down and lat_up", MoeBlock, {**w, "lat_down": bf16(32, 64)}, 2)
    raises("no projection for the adapters", MoeBlock, w, 2, adapters={"lat_up": ()})
    latent = {**w, "lat_down": bf16(32, 64), "lat_up": bf16(64, 32)}
    raises("no projection for the adapters", MoeBlock, latent, 2, adapters={"router": ()})


def test_moe_block_refuses_weights_that_it_would_drop(capi, monkeypatch):
    from int4_routed_expert_fp32_gb300.block import MoeBlock
    monkeypatch.setattr(capi, "router_prepare", lambda w: None)
    w = {n: f32(1) for n in capi.EXPERT_NAMES}
    w["router_w"] = f32(16, 64)
    assert MoeBlock({**w, "router_bias": None, "shared_gate": None}, 2).shared is None
    raises("unknown weight names: .*'shared_gate_w'", MoeBlock, {**w, "shared_gate_w": None}, 2)
    raises("lat_norm belongs to", MoeBlock, {**w, "lat_norm": bf16(32)}, 2)
    raises("come together", MoeBlock, {**w, "shared_gate": bf16(32, 64)}, 2)
    raises("come together", MoeBlock, {**w, "shared_gate": bf16(32, 64),
                                       "shared_up": bf16(32, 64)}, 2)
    raises("router_w is required", MoeBlock, {n: w[n] for n in capi.EXPERT_NAMES}, 2)
    terms = bf16(3, 16, 64)
    assert MoeBlock({**w, "router_w_terms": terms}, 2).w_terms is terms


def test_adapter_stall_selftest_refusals(capi):
    L, n = capi.lib, capi.launch_count()
    bad, uns = capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED

    def call(T=9, R=8, kernel=1, stage=0, limit=20_000_000, x=FAKE, ws_bytes=1 << 30):
        return L.moe_adapter_linear_stall_selftest(x, FAKE, FAKE, FAKE, FAKE, None, T, 64, 24, R, 3,
                                                   kernel, stage, limit, FAKE, FAKE, ws_bytes,
                                                   None)

    for kw in (dict(kernel=-1), dict(kernel=3), dict(stage=-1), dict(limit=999),
               dict(limit=5_000_000_001), dict(x=None), dict(T=-1)):
        assert call(**kw) == bad, kw
    for kw in (dict(T=1, R=16, kernel=0), dict(T=300, kernel=2), dict(R=12)):
        assert call(**kw) == uns, kw
    assert call(ws_bytes=0) == capi.MOE_ERR_WORKSPACE
    assert capi.launch_count() == n


def test_adapter_linear_refuses_overlapping_memory(capi):
    """CTAs write y while others read the inputs: y over any of them, or the workspace
    over any, is refused (adjacent memory is not)."""
    T, K, N, R, n = 9, 64, 64, 8, 3
    sizes = dict(x=T * K * 2, w=N * K * 2, a=n * R * K * 2, b=n * N * R * 2, ids=T * 4,
                 scale=n * 4, y=T * N * 2, ws=int(capi.lib.moe_adapter_linear_workspace_size(
                     T, K, N, R)))
    apart = {name: FAKE * (i + 1) for i, name in enumerate(sizes)}
    n0 = capi.launch_count()

    def call(**at):
        p = {**apart, **at}
        return capi.lib.moe_adapter_linear(p["x"], p["w"], p["a"], p["b"], p["ids"], p["scale"],
                                           T, K, N, R, n, p["y"], p["ws"], sizes["ws"], None)

    for name in sizes:
        if name == "y":
            continue
        step = 256 if name == "ws" else 16
        for y in (apart[name], apart[name] + (sizes[name] - 1) // step * step,
                  apart[name] - (sizes["y"] - 1) // step * step):
            assert call(y=y) == capi.MOE_ERR_INVALID, (name, y)
        if name != "ws":
            assert call(ws=apart[name]) == capi.MOE_ERR_INVALID, name
    x = bf16(T, K)
    w, a, b, ids = bf16(N, K), bf16(n, R, K), bf16(n, N, R), torch.zeros(T, dtype=torch.int32)
    raises("out must not share memory with x", capi.adapter_linear, x, w, a, b, ids, out=x)
    raises("out must not share memory with w", capi.adapter_linear, x, w, a, b, ids, out=w[5:5 + T])
    both = bf16(2 * T, K)
    raises(CUDA_ONLY, capi.adapter_linear, both[:T], w, a, b, ids, out=both[T:])
    assert capi.launch_count() == n0


def test_adapter_linear_refuses_more_tokens_or_columns_than_a_grid_has(capi):
    L, n = capi.lib, capi.launch_count()
    far = 1 << 50   # apart from FAKE by more than any of these tensors is long

    def call(T, N):
        return L.moe_adapter_linear(FAKE, FAKE, FAKE, FAKE, FAKE, None, T, 64, N, 8, 3, far,
                                    2 * far, 1 << 40, None)

    for T, N in ((65535 * 128 + 1, 24), (2 ** 31 - 1, 24), (9, 65535 * 128 + 8)):
        assert call(T, N) == capi.MOE_ERR_UNSUPPORTED, (T, N)
    assert capi.launch_count() == n


def test_adapter_linear_of_a_few_tokens_needs_no_workspace(capi):
    """One launch up to four tokens of T R <= 64; above, the low-rank vectors of a launch
    of their own."""
    size = capi.lib.moe_adapter_linear_workspace_size
    for T, R in ((1, 8), (1, 64), (2, 32), (4, 16)):
        assert size(T, 7168, 3584, R) == 0, (T, R)
    for T, R in ((1, 72), (2, 40), (4, 24), (5, 8), (8, 8), (9, 8)):
        assert size(T, 7168, 3584, R) >= T * R * 4, (T, R)


def test_c_entries_keep_no_containers_that_throw():
    """What a launch keeps sits in tables of fixed size: an exception would leave the
    C entry."""
    import glob
    import os
    from tests.test_tensor_memory_rule import CSRC
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = f.read()
        for name in ("std::vector", "std::map", "std::unordered_map", "std::string",
                     "std::function"):
            assert name not in text, (os.path.basename(path), name)
