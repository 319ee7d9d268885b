"""Refusals of the operators for a few tokens: by the Python binding on host tensors, and
by the C entry points before any launch (no GPU needed)."""
import ctypes

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


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def raises(match, fn, *args, **kwargs):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kwargs)


def experts(E=4, D=64, I=128):
    w = {}
    for name, N, K in (("gate", I, D), ("up", I, D), ("down", D, I)):
        w[name + "_packed"], w[name + "_scale"] = i32(E, N, K // 8), bf16(E, N, K // 32)
    return w


def layer(E=4, H=64, I=128, L=0, S=0):
    w = dict(experts(E, L or H, I), router_w=f32(E, H), router_bias=f32(E))
    if L:
        w.update(lat_down=bf16(L, H), lat_up=bf16(H, L), lat_norm=bf16(L))
    if S:
        w.update(shared_gate=bf16(S, H), shared_up=bf16(S, H), shared_down=bf16(H, S))
    return w


# ---------------------------------------------------------------- the binding

def test_matvec_binding(capi):
    f = capi.int4_matvec
    raises(CUDA_ONLY, f, bf16(2, 64), i32(8, 8), bf16(8, 2))
    raises(CUDA_ONLY, f, bf16(2, 72)[:, :64], i32(8, 8), bf16(8, 2))
    raises(CUDA_ONLY, f, bf16(2, 64), i32(8, 8), bf16(8, 2), out=bf16(2, 8))
    raises("x: expected torch.bfloat16", f, f32(2, 64), i32(8, 8), bf16(8, 2))
    raises("x: expected shape", f, bf16(64), i32(8, 8), bf16(8, 2))
    raises("x: its rows", f, bf16(64, 2).t(), i32(8, 8), bf16(8, 2))
    raises("x: its rows", f, bf16(1, 64).expand(2, 64), i32(8, 8), bf16(8, 2))
    raises("w_packed: expected shape", f, bf16(2, 64), i32(8, 9), bf16(8, 2))
    raises("w_packed: expected shape", f, bf16(2, 64), i32(1, 8, 8), bf16(8, 2))
    raises("w_packed: expected torch.int32", f, bf16(2, 64), i32(8, 8).long(), bf16(8, 2))
    raises("w_packed must be contiguous", f, bf16(2, 64), i32(8, 16)[:, :8], bf16(8, 2))
    raises("w_scale: expected shape", f, bf16(2, 64), i32(8, 8), bf16(8, 3))
    raises("out: expected shape", f, bf16(2, 64), i32(8, 8), bf16(8, 2), out=bf16(2, 9))


def test_experts_binding(capi):
    f, w = capi.experts_few, experts()
    idx, p, x = i32(3, 2), f32(3, 2), bf16(3, 64)
    raises(CUDA_ONLY, f, idx, p, x, w)
    raises(CUDA_ONLY, f, idx, p, x, dict(w, other=bf16(1)))
    raises("x: expected torch.bfloat16", f, idx, p, x.float(), w)
    raises("x must be contiguous", f, idx, p, bf16(3, 128)[:, :64], w)
    raises("topk_idx: expected shape", f, i32(4, 2), p, x, w)
    raises("topk_idx: expected torch.int32", f, idx.long(), p, x, w)
    raises("topk_w: expected shape", f, idx, f32(3, 3), x, w)
    raises("down_scale is required", f, idx, p, x, {n: t for n, t in w.items() if n != "down_scale"})
    raises("up_packed: expected shape", f, idx, p, x, dict(w, up_packed=i32(4, 128, 9)))
    raises("out: expected torch.bfloat16", f, idx, p, x, w, out=f32(3, 64))
    raises("must not share memory with x|" + CUDA_ONLY, f, idx, p, x, w, out=x)


def test_layer_binding(capi):
    f, x = capi.layer_few, bf16(3, 64)
    raises(CUDA_ONLY, f, x, layer(), 2)
    raises(CUDA_ONLY, f, x, layer(L=192, S=64), 2)
    raises("x: expected shape", f, bf16(64), layer(), 2)
    raises("unknown weight names", f, x, dict(layer(), gate=bf16(1)), 2)
    raises("router_w: expected shape", f, bf16(3, 128), layer(), 2)
    raises("lat_up is required", f, x, {n: t for n, t in layer(L=64).items() if n != "lat_up"}, 2)
    raises("lat_up needs lat_down", f, x, dict(layer(), lat_up=bf16(64, 64)), 2)
    raises("shared_up needs shared_gate", f, x, dict(layer(), shared_up=bf16(64, 64)), 2)
    with pytest.raises(TypeError):
        f(x, layer(), 2.5)


# ---------------------------------------------------------------- the C entries

def matvec_args(**kw):
    a = dict(x=FAKE, x_ld=64, w=FAKE << 4, s=FAKE << 5, T=2, N=8, K=64, y=FAKE << 6, stream=None)
    a.update(kw)
    return a.values()


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "INVALID"), (dict(N=0), "INVALID"), (dict(K=0), "INVALID"),
    (dict(x_ld=32), "INVALID"), (dict(x=None), "INVALID"), (dict(w=None), "INVALID"),
    (dict(s=None), "INVALID"), (dict(y=None), "INVALID"), (dict(x=FAKE + 8), "INVALID"),
    (dict(w=FAKE + 4), "INVALID"), (dict(s=FAKE + 2), "INVALID"), (dict(y=FAKE + 1), "INVALID"),
    (dict(y=FAKE + 64), "INVALID"), (dict(y=(FAKE << 4) + 32), "INVALID"),
    (dict(y=(FAKE << 5) + 30), "INVALID"), (dict(T=17), "UNSUPPORTED"),
    (dict(K=48), "UNSUPPORTED"), (dict(x_ld=68), "UNSUPPORTED"),
    (dict(K=(1 << 20) + 32, x_ld=1 << 21), "UNSUPPORTED"), (dict(N=(1 << 30) + 1), "UNSUPPORTED"),
])
def test_matvec_refusals(capi, kw, code):
    n = capi.launch_count()
    assert capi.lib.moe_int4_matvec(*matvec_args(**kw)) == getattr(capi, "MOE_ERR_" + code)
    assert capi.launch_count() == n


def test_matvec_of_no_rows(capi):
    assert capi.lib.moe_int4_matvec(*matvec_args(T=0, x=None, y=None)) == capi.MOE_OK


def experts_args(capi, **kw):
    a = dict(x=FAKE, idx=FAKE << 1, p=FAKE << 2, T=3, D=64, E=4, k=2, I=128, g=FAKE << 4,
             gs=FAKE << 5, u=FAKE << 6, us=FAKE << 7, d=FAKE << 8, ds=FAKE << 9, out=FAKE << 10,
             ws=FAKE << 11, bytes=1 << 22, stream=None)
    a.update(kw)
    return list(a.values())


SIZES = [(dict(T=-1), "INVALID"), (dict(D=0), "INVALID"), (dict(E=0), "INVALID"),
         (dict(k=0), "INVALID"), (dict(I=0), "INVALID"), (dict(T=33), "UNSUPPORTED"),
         (dict(D=96), "UNSUPPORTED"), (dict(I=96), "UNSUPPORTED"), (dict(E=2049), "UNSUPPORTED"),
         (dict(k=5), "UNSUPPORTED"), (dict(E=64, k=33), "UNSUPPORTED"),
         (dict(D=(1 << 20) + 64), "UNSUPPORTED"), (dict(I=(1 << 20) + 64), "UNSUPPORTED")]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(x=None), "INVALID"), (dict(idx=None), "INVALID"), (dict(p=None), "INVALID"),
    (dict(g=None), "INVALID"), (dict(ds=None), "INVALID"), (dict(out=None), "INVALID"),
    (dict(ws=None), "INVALID"), (dict(x=FAKE + 8), "INVALID"), (dict(u=(FAKE << 6) + 8), "INVALID"),
    (dict(us=(FAKE << 7) + 2), "INVALID"), (dict(idx=FAKE + 2), "INVALID"),
    (dict(out=(FAKE << 10) + 8), "INVALID"), (dict(ws=(FAKE << 11) + 128), "INVALID"),
    (dict(out=FAKE), "INVALID"), (dict(out=FAKE << 8), "INVALID"), (dict(ws=FAKE << 4), "INVALID"),
    (dict(out=FAKE << 11), "INVALID"), (dict(bytes=1024), "WORKSPACE"),
])
def test_experts_refusals(capi, kw, code):
    n, want = capi.launch_count(), getattr(capi, "MOE_ERR_" + code)
    assert capi.lib.moe_experts_few(*experts_args(capi, **kw)) == want
    args = experts_args(capi, **kw)
    args[14:14] = [0, 10 ** 6]
    assert capi.lib.moe_experts_few_stall_selftest(*args) == want
    assert capi.launch_count() == n


def test_experts_without_tokens(capi):
    L = capi.lib
    assert L.moe_experts_few(*experts_args(capi, T=0, x=None, ws=None)) == capi.MOE_OK
    assert L.moe_experts_few_workspace_size(0, 64, 4, 2, 128) == 0
    assert L.moe_experts_few_workspace_size(33, 64, 4, 2, 128) == 0
    assert L.moe_experts_few_workspace_size(3, 64, 4, 2, 128) > 0
    for stage, limit in ((-1, 10 ** 6), (0, 999), (0, 6 * 10 ** 9)):
        args = experts_args(capi)
        args[14:14] = [stage, limit]
        assert L.moe_experts_few_stall_selftest(*args) == capi.MOE_ERR_INVALID


WEIGHTS = ("router_w", "router_bias", "gate_packed", "gate_scale", "up_packed", "up_scale",
           "down_packed", "down_scale", "lat_down", "lat_up", "lat_norm", "shared_gate",
           "shared_up", "shared_down")


def layer_call(capi, cfg=None, weights=None, x=FAKE, out=FAKE << 20, ws=FAKE << 21, size=1 << 24):
    c = dict(T=3, H=64, E=4, k=2, I=128, L=64, act_bits=16, renorm=1, eps=1e-6, I_shared=64)
    c.update(cfg or {})
    w = {n: FAKE << (i + 1) for i, n in enumerate(WEIGHTS)}
    w.update(weights or {})
    names = [n for n, _ in capi.MoeWeights._fields_]
    return capi.lib.moe_layer_few(ctypes.byref(capi.MoeConfig(*c.values())),
                                  ctypes.byref(capi.MoeWeights(*[w.get(n) for n in names])), x, out,
                                  ws, size, None)


@pytest.mark.parametrize("kw,code", [(dict(s, **({"L": 0, "H": s["D"]} if "D" in s else {})), c)
                                     for s, c in SIZES] + [
    (dict(H=0), "INVALID"), (dict(L=-64), "INVALID"), (dict(I_shared=-1), "INVALID"),
    (dict(eps=-1.0), "INVALID"), (dict(eps=float("nan")), "INVALID"), (dict(H=96), "UNSUPPORTED"),
    (dict(L=32), "UNSUPPORTED"),
    (dict(H=(1 << 20) + 64), "UNSUPPORTED"), (dict(L=(1 << 20) + 64), "UNSUPPORTED"),
    (dict(I_shared=(1 << 20) + 64), "UNSUPPORTED"), (dict(I_shared=32), "UNSUPPORTED"),
    (dict(act_bits=8), "UNSUPPORTED")])
def test_layer_size_refusals(capi, kw, code):
    n = capi.launch_count()
    kw = {a: b for a, b in kw.items() if a != "D"}
    assert layer_call(capi, kw) == getattr(capi, "MOE_ERR_" + code)
    c = dict(T=3, H=64, E=4, k=2, I=128, L=64, act_bits=16, renorm=1, eps=1e-6, I_shared=64)
    c.update(kw)
    assert capi.lib.moe_layer_few_workspace_size(ctypes.byref(capi.MoeConfig(*c.values()))) == 0
    assert capi.launch_count() == n


def test_layer_pointer_refusals(capi):
    n, bad = capi.launch_count(), capi.MOE_ERR_INVALID
    for name in WEIGHTS:
        if name != "lat_norm":
            assert layer_call(capi, weights={name: None}) == bad, name
        assert layer_call(capi, weights={name: (FAKE << 25) + 1}) == bad, name
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(x=FAKE + 2), dict(out=FAKE + 2),
               dict(ws=(FAKE << 21) + 16), dict(out=FAKE), dict(out=FAKE << 9), dict(ws=FAKE << 14),
               dict(out=FAKE << 21)):
        assert layer_call(capi, **kw) == bad, kw
    assert layer_call(capi, size=256) == capi.MOE_ERR_WORKSPACE
    assert layer_call(capi, dict(T=0), x=None, out=None, ws=None) == capi.MOE_OK
    assert capi.lib.moe_layer_few(None, None, FAKE, FAKE, FAKE, 0, None) == bad
    assert capi.lib.moe_layer_few_workspace_size(None) == 0
    assert capi.launch_count() == n


def test_layer_object(capi, monkeypatch):
    """forward_few hands on the layer's own weights and sizes with the call's tokens, and
    refuses 8-bit activations, another width and host tensors."""
    L = capi.MoeLayer.__new__(capi.MoeLayer)
    L.wstruct, L.device = capi.MoeWeights(), torch.device("cpu")
    L.cfg = capi.MoeConfig(100, 64, 4, 2, 128, 64, 16, 0, 1e-5, 64)
    raises(CUDA_ONLY, L.forward_few, bf16(3, 64))
    raises("x: expected shape", L.forward_few, bf16(3, 128))
    raises("out: expected shape", L.forward_few, bf16(3, 64), out=bf16(100, 64))
    seen = []
    monkeypatch.setattr(capi, "_device_of", lambda *a: torch.device("cpu"))
    monkeypatch.setattr(capi, "_layer_few", lambda cfg, w, x, out, dev: seen.append((cfg, w, out)))
    L.forward_few(bf16(3, 64))
    cfg, w, out = seen[0]
    got = [getattr(cfg, n) for n, _ in capi.MoeConfig._fields_]
    want = [getattr(L.cfg, n) for n, _ in capi.MoeConfig._fields_]
    assert cfg.T == 3 and got[1:] == want[1:] and w is L.wstruct and out.shape == (3, 64)
    L.cfg.act_bits = 8
    raises("act_bits 16", L.forward_few, bf16(3, 64))
