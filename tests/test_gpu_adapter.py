"""GPU parity of the adapter projection against a 64-bit reference.

Tolerance.  One rounding to bf16 is at most 2^-8 of the value.  Before it, fp32
sums of K products err by at most (K / 16 + 16) 2^-24 of the sum of their
magnitudes, about sqrt(K) of a typical value's, and the low-rank vector is kept
to 16 bits: 2^-16 of the sum of |s p_j B_j|.  With these inputs both sums of
magnitudes are within 100 times the norm of the two terms, so 1e-3 of the
row's RMS bounds them with room.
"""
import numpy as np
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


def inputs(T, K, N, R, n, ids, seed, scaled=True):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, std):
        return (std * torch.randn(*shape, generator=g)).to(BF16).to(DEV)

    if isinstance(ids, str):
        r = np.random.default_rng(seed)
        if ids == "mixed":       # any adapter anywhere, a few rows without
            v = r.integers(-1, n, size=T)
        elif ids == "runs":      # requests of consecutive tokens
            v = np.repeat(r.integers(-1, n, size=T), r.integers(1, 90, size=T))[:T]
        elif ids == "none":
            v = np.full(T, -1)
        else:                    # one adapter for all
            v = np.full(T, n - 1)
        ids = torch.from_numpy(v.astype(np.int32))
    scale = (0.5 + torch.rand(n, generator=g)).to(DEV) if scaled else None
    return (randn(T, K, std=1.0), randn(N, K, std=0.02), randn(n, R, K, std=0.02),
            randn(n, N, R, std=0.1), ids.to(torch.int32).to(DEV), scale)


def ref(x, w, a, b, ids, scale):
    x, w, a, b = (t.double() for t in (x, w, a, b))
    y = x @ w.T
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i).flatten()
        if len(rows):
            low = x[rows] @ a[i].T @ b[i].T
            y[rows] += low if scale is None else low * scale[i].double()
    return y


def check(moe, args, what=""):
    got = moe.adapter_linear(*args)
    assert moe.check_error() == 0
    want = ref(*args)
    err = (got.double() - want).abs()
    rms = want.square().mean(dim=1, keepdim=True).sqrt()
    assert torch.all(err <= 2.0 ** -8 * want.abs() + 1e-3 * rms), \
        (what, float((err / rms.clamp_min(1e-30)).max()))
    return got


SHAPES = [  # T, K, N, R, adapters
    (1, 256, 128, 16, 1), (1, 32, 8, 8, 2), (2, 64, 136, 24, 5), (7, 1056, 264, 8, 3),
    (16, 512, 520, 16, 9), (17, 512, 72, 40, 4), (33, 2048, 384, 16, 33), (64, 224, 1000, 64, 7),
    (65, 416, 256, 128, 3), (127, 256, 640, 16, 60), (128, 256, 128, 16, 128),
    (129, 256, 128, 8, 200), (200, 992, 328, 48, 12), (256, 512, 256, 16, 16),
    (257, 512, 264, 32, 6), (600, 736, 520, 16, 5), (1000, 256, 1032, 64, 3),
    (1500, 320, 768, 72, 4), (2049, 128, 512, 16, 40), (300, 7168, 256, 16, 4),
    # many output tiles to a CTA pair, with one to a few K steps each
    (4100, 64, 5000, 16, 30), (4100, 32, 4104, 48, 3), (3000, 512, 4600, 128, 9),
]


@pytest.mark.parametrize("ids", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_adapter_linear(moe, shape, ids):
    T, K, N, R, n = shape
    check(moe, inputs(T, K, N, R, n, ids, T + K + N, scaled=ids != "runs"), (shape, ids))


@pytest.mark.parametrize("T", [1, 40, 300, 700])
def test_rows_without_an_adapter_are_the_projection(moe, T):
    """ids of -1 give the projection's own bits whatever the other rows use,
    and never read an adapter (theirs hold NaN here)."""
    x, w, a, b, ids, scale = inputs(T, 512, 264, 16, 4, "mixed", 3)
    a[2] = float("nan")
    b[2] = float("nan")
    ids[ids == 2] = -1
    alone = moe.adapter_linear(x, w, a, b, torch.full_like(ids, -1), scale)
    both = moe.adapter_linear(x, w, a, b, ids, scale)
    assert torch.equal(both[ids < 0], alone[ids < 0])
    assert not torch.isnan(both).any()
    check(moe, (x, w, a[:2], b[:2], torch.where(ids > 1, -1, ids), scale[:2]))


@pytest.mark.parametrize("T", [3, 300, 700])
def test_infinities_and_nan_stay_in_their_row(moe, T):
    x, w, a, b, ids, scale = inputs(T, 256, 136, 16, 3, "mixed", 6)
    clean = moe.adapter_linear(x, w, a, b, ids, scale)
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    got = moe.adapter_linear(x, w, a, b, ids, scale)
    rest = [0] + list(range(3, T))
    assert torch.equal(got[rest], clean[rest])
    assert not torch.isfinite(got[1]).any() and torch.isnan(got[2]).all()


@pytest.mark.parametrize("T", [5, 400, 900])
def test_ids_out_of_range_select_none_and_are_reported(moe, T):
    x, w, a, b, ids, scale = inputs(T, 256, 136, 16, 3, "mixed", 8)
    want = moe.adapter_linear(x, w, a, b, ids, scale)
    assert moe.check_error() == 0
    bad = ids.clone()
    bad[ids < 0] = 3
    bad[(ids < 0) & (torch.arange(T, device=DEV) % 2 == 0)] = -2147483648
    assert (bad != ids).any()
    got = moe.adapter_linear(x, w, a, b, bad, scale)
    assert moe.check_error() == moe.capi.MOE_ERR_INVALID
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 64, 300, 1000])
def test_same_bits_again_on_another_stream_and_from_a_graph(moe, T):
    args = inputs(T, 512, 520, 16, 6, "mixed", 11)
    want = moe.adapter_linear(*args)
    torch.cuda.synchronize()
    n0 = moe.launch_count()
    assert torch.equal(moe.adapter_linear(*args), want)
    assert moe.launch_count() - n0 == (1 if T * args[2].shape[1] <= 64 else 2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [moe.adapter_linear(*args) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)
    x = torch.zeros_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.adapter_linear(x, *args[1:])
    x.copy_(args[0])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert moe.check_error() == 0


@pytest.mark.parametrize("T", [3, 130, 700])
def test_writes_stay_inside_output_and_workspace(moe, T):
    K, N, R, n = 288, 200, 24, 5
    x, w, a, b, ids, scale = inputs(T, K, N, R, n, "mixed", 13)
    want = moe.adapter_linear(x, w, a, b, ids, scale)
    guard = 1 << 12
    need = int(moe.lib.moe_adapter_linear_workspace_size(T, K, N, R))
    ws = torch.full((need + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((T * N * 2 + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    rc = moe.lib.moe_adapter_linear(
        x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(), ids.data_ptr(), scale.data_ptr(),
        T, K, N, R, n, out.data_ptr() + guard, ws.data_ptr() + guard, need,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and moe.check_error() == 0
    for buf in (ws, out):
        assert torch.all(buf[:guard] == 0xA5) and torch.all(buf[-guard:] == 0xA5)
    assert torch.equal(out[guard:-guard].view(BF16).reshape(T, N), want)


def test_adapter_offsets_pass_32_bits(moe):
    """The last of 80 adapters begins past 2^31 elements of lora_a (zeros but
    for that one)."""
    T, K, N, R, n = 4, 256 * 1024, 16, 128, 80
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.zeros(n, R, K, dtype=BF16, device=DEV)
    a[n - 1] = 0.02 * torch.randn(R, K, generator=g, device=DEV)
    b = (0.1 * torch.randn(n, N, R, generator=g, device=DEV)).to(BF16)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF16)
    w = (0.02 * torch.randn(N, K, generator=g, device=DEV)).to(BF16)
    ids = torch.tensor([n - 1, 0, -1, n - 1], dtype=torch.int32, device=DEV)
    got = moe.adapter_linear(x, w, a, b, ids)
    assert moe.check_error() == 0
    want = x.double() @ w.double().T
    for t in (0, 3):
        want[t] += x[t].double() @ a[n - 1].double().T @ b[n - 1].double().T
    rms = want.square().mean(dim=1, keepdim=True).sqrt()
    assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3 * rms)


@pytest.mark.parametrize("R", [16, 40, 128])
@pytest.mark.parametrize("T", [40, 300, 1500])
def test_an_adapter_that_is_not_finite_reaches_its_own_tokens_only(moe, T, R):
    """Infinities and NaN in lora_b (some columns) and lora_a of one adapter:
    tokens of the others keep their bits, its own have the formula's values."""
    K, N, n = 256, 520, 5
    x, w, a, b, ids, scale = inputs(T, K, N, R, n, "mixed", 17)
    clean = moe.adapter_linear(x, w, a, b, ids, scale)
    assert moe.check_error() == 0
    b[2, 7, R - 1] = float("nan")
    b[2, 300, 0] = float("inf")
    b[2, 519, 3] = -float("inf")
    got = moe.adapter_linear(x, w, a, b, ids, scale)
    assert moe.check_error() == 0
    own = ids == 2
    assert torch.equal(got[~own], clean[~own])
    cols = torch.tensor([c not in (7, 300, 519) for c in range(N)], device=DEV)
    assert torch.equal(got[own][:, cols], clean[own][:, cols])
    want = ref(x, w, a, b, ids, scale)[own][:, [7, 300, 519]]
    bad = got[own][:, [7, 300, 519]].double()
    assert torch.isnan(bad[:, 0]).all()
    assert torch.equal(bad[:, 1:], want[:, 1:])      # +inf or -inf, by p's sign
    a[2] = float("nan")
    got = moe.adapter_linear(x, w, a, b, ids, scale)
    assert torch.equal(got[~own], clean[~own]) and torch.isnan(got[own]).all()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T", [1, 4, 40, 100, 200, 700])
def test_calls_that_depend_on_one_another(moe, T, graph):
    """Each call's x is the output of the one before, and its ids and scale are written
    just ahead of it: the kernels of a call may start before those of the call before
    have ended, and read nothing that is not complete."""
    R, n, steps = 16, 5, 6
    widths = [2048, 1024, 2048, 512, 1056, 2048, 256]
    g = torch.Generator().manual_seed(T)
    layers, wanted = [], []
    for i in range(steps):
        K, N = widths[i], widths[i + 1]
        x, w, a, b, ids, scale = inputs(T, K, N, R, n, "mixed", 40 + i)
        layers.append((w, a, b, ids, scale))
    x0 = torch.randn(T, widths[0], generator=g).to(BF16).to(DEV)
    h = x0
    for w, a, b, ids, scale in layers:
        torch.cuda.synchronize()
        h = moe.adapter_linear(h, w, a, b, ids, scale)
        torch.cuda.synchronize()
        wanted.append(h)
    idle = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    now, s = idle.clone(), torch.zeros(n, device=DEV)

    def chain():
        out, h = [], x0
        for w, a, b, ids, scale in layers:
            now.copy_(ids)
            s.copy_(scale)
            h = moe.adapter_linear(h, w, a, b, now, s)
            out.append(h)
        now.copy_(idle)
        s.zero_()
        return out

    got = chain()
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = chain()
        for _ in range(20):
            captured.replay()
    else:
        for _ in range(20):
            got = chain()
    torch.cuda.synchronize()
    assert moe.check_error() == 0
    for i, (a, b) in enumerate(zip(got, wanted)):
        assert torch.equal(a, b), i
