"""The training operators on a B200, through the C ABI, against the formulas in
64 bits.

Tolerances count roundings. An fp32 sum of n products is off by at most
n 2^-23 sum|a b| (one step of the running sum per addition, truncated or
rounded); a bf16 result by half a step, 2^-8 |value|. In the gated gradient the
exponential, the quotient and the products after it are each good to a few
2^-24, counted as 2^-18 (1 + |g|) of d u. An orthogonalised update rounds three
operands a step to fp16 (half a step is 2^-11 of the value), and each turns X by
at most about its own size, so its error is at most steps * 3 * 2^-11 of the
result's norm, beside the result's own 2^-8."""
import math

import numpy as np
import pytest

from helpers import Guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_tcgen05_b200 as moe  # noqa: E402

ACTS = {moe.MOE_EPILOGUE_NONE: None, moe.MOE_EPILOGUE_SWIGLU: "silu", moe.MOE_EPILOGUE_GEGLU: "gelu",
        moe.MOE_EPILOGUE_REGLU: "relu"}
COEFFS = (3.4445, -4.7750, 2.0315)
BF16 = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _ws(n=1 << 20):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def act64(kind, g):
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if kind == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return torch.clamp(g, min=0), (g > 0).double()


def within(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}, largest excess "
                           f"{((got - ref).abs() - tol)[bad].max().item():.3e}")


def rows64(dC, B, counts):
    """d = dC B per expert and the bound of its fp32 sums, both fp64."""
    d = torch.zeros(dC.shape[0], B.shape[2], dtype=torch.float64, device="cuda")
    s = torch.zeros_like(d)
    r = 0
    for e, c in enumerate(counts):
        d[r:r + c] = dC[r:r + c].double() @ B[e].double()
        s[r:r + c] = dC[r:r + c].double().abs() @ B[e].double().abs()
        r += c
    return d, s * dC.shape[1] * 2.0**-23


# rows per expert, N, K
GROUPS = [
    ([1], 128, 128),
    ([3, 0, 5], 256, 128),
    ([0, 0, 16, 0], 128, 384),
    ([17, 64, 1, 0, 33], 384, 256),
    ([127, 128, 129], 128, 640),
    ([0, 300, 0, 77, 255, 1], 512, 384),
    ([640, 2, 0, 500], 1152, 896),
    ([1] * 40, 128, 256),
    ([2100], 256, 256),
    ([1, 0, 2, 0] * 256, 128, 128),  # 1024 experts
    ([1100, 1300, 0, 1500, 700, 1, 1900, 1692], 1024, 4992),  # pairs of SMs and their last rows
]


@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("with_h", [True, False])
def test_dgrad(counts, N, K, act, with_h):
    if ACTS[act] is None and with_h:
        with_h = False
    E, R, behind = len(counts), sum(counts), 5
    M = R + behind
    gen = _gen(R * 7 + N + K + act)
    dC, B = _randn(gen, M, N), _randn(gen, E, N, K, std=0.05)
    dC[R:] = float("nan")  # rows of no expert
    gated = ACTS[act] is not None
    gu = _randn(gen, M, 2 * K, std=2.0) if gated else None
    out = Guarded((M, 2 * K if gated else K), BF16, fill=0x7B)
    h = Guarded((M, K), BF16, fill=0x7B) if with_h else None
    ws = _ws()
    before = out.t[R:].clone()
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets(counts), M, E, N, K, act, out.t, gu=gu,
                               h=h.t if with_h else None, ws=ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0
    assert out.intact() and torch.equal(out.t[R:].view(torch.int16), before.view(torch.int16))
    d, eps = rows64(dC[:R], B, counts)
    if not gated:
        within(out.t[:R], d, d.abs() * 2.0**-8 + eps, "dA")
        return
    g, u = gu[:R, :K].double(), gu[:R, K:].double()
    a, da = act64(ACTS[act], g)
    slack = 2.0**-18 * (1 + g.abs()) * (d * u).abs()
    ref = d * u * da
    within(out.t[:R, :K], ref, ref.abs() * 2.0**-8 + eps * (u * da).abs() + slack, "gate gradient")
    ref = d * a
    within(out.t[:R, K:], ref, ref.abs() * 2.0**-8 + eps * a.abs() + 2.0**-18 * (1 + g.abs()) * (d * g).abs(),
           "up gradient")
    if with_h:
        assert h.intact()
        ref = a * u
        within(h.t[:R], ref, ref.abs() * 2.0**-8 + 2.0**-18 * (1 + g.abs()) * (g * u).abs(), "h")


@pytest.mark.parametrize("act", [moe.MOE_EPILOGUE_NONE, moe.MOE_EPILOGUE_SWIGLU])
@pytest.mark.parametrize("counts", [[1, 0, 9, 16], [0, 33, 64, 5], [70, 1, 0, 130], [257, 31, 32, 33], [511, 513],
                                    [48, 240, 250, 272], [2049, 15], [4200],
                                    [200, 0, 0, 0, 1, 3, 0, 0], [0, 65, 0, 0, 31, 33, 64]])
def test_dgrad_row_tiles(counts, act):
    """Row counts around the sizes that tiles, their groups of rows and the small boxes end at."""
    E, R, N, K = len(counts), sum(counts), 640, 384
    gen = _gen(R + act)
    dC, B = _randn(gen, R, N), _randn(gen, E, N, K, std=0.05)
    gated = act != moe.MOE_EPILOGUE_NONE
    gu = _randn(gen, R, 2 * K) if gated else None
    out = torch.full((R, 2 * K if gated else K), float("nan"), dtype=BF16, device="cuda")
    h = torch.full((R, K), float("nan"), dtype=BF16, device="cuda") if gated else None
    ws = _ws(1 << 22)
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets(counts), R, E, N, K, act, out, gu=gu, h=h, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    d, eps = rows64(dC, B, counts)
    if not gated:
        within(out, d, d.abs() * 2.0**-8 + eps, "dA")
        return
    g, u = gu[:, :K].double(), gu[:, K:].double()
    a, da = act64("silu", g)
    ref = torch.cat([d * u * da, d * a], 1)
    tol = ref.abs() * 2.0**-8 + torch.cat([eps * (u * da).abs(), eps * a.abs()], 1) + 2.0**-18 * torch.cat(
        [(1 + g.abs()) * (d * u).abs(), (1 + g.abs()) * (d * g).abs()], 1)
    within(out, ref, tol, "gated gradients")
    within(h, a * u, (a * u).abs() * 2.0**-8 + 2.0**-18 * (1 + g.abs()) * (g * u).abs(), "h")


@pytest.mark.parametrize("act", [moe.MOE_EPILOGUE_SWIGLU, moe.MOE_EPILOGUE_GEGLU, moe.MOE_EPILOGUE_REGLU])
def test_dgrad_activation_far_from_zero(act):
    """Gates of both signs up to 100, zeros included: no overflow, relu' (0) = 0."""
    R, N, K = 8, 128, 128
    gen = _gen(3)
    dC, B = _randn(gen, R, N), _randn(gen, 1, N, K, std=0.05)
    gu = _randn(gen, R, 2 * K)
    gu[0, :K], gu[1, :K], gu[2, :K], gu[3, :K], gu[4, :K] = 100.0, -100.0, 0.0, -8.0, 12.0
    out = torch.empty(R, 2 * K, dtype=BF16, device="cuda")
    h = torch.empty(R, K, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets([R]), R, 1, N, K, act, out, gu=gu, h=h, ws=_ws())
    d, eps = rows64(dC, B, [R])
    g, u = gu[:, :K].double(), gu[:, K:].double()
    a, da = act64(ACTS[act], g)
    assert torch.isfinite(out).all() and torch.isfinite(h).all()
    ref = torch.cat([d * u * da, d * a], 1)
    tol = ref.abs() * 2.0**-8 + torch.cat([eps * (u * da).abs(), eps * a.abs()], 1) + 2.0**-18 * torch.cat(
        [(1 + g.abs()) * (d * u).abs(), (1 + g.abs()) * (d * g).abs()], 1)
    within(out, ref, tol, "gated gradients")
    if act == moe.MOE_EPILOGUE_REGLU:
        assert (out[2] == 0).all() and (h[2] == 0).all()


def weights64(dC, A, counts):
    E, N, K = len(counts), dC.shape[1], A.shape[1]
    d = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    s = torch.zeros_like(d)
    r = 0
    for e, c in enumerate(counts):
        x, y = dC[r:r + c].double(), A[r:r + c].double()
        d[e] = x.T @ y
        s[e] = (x.abs().T @ y.abs()) * max(c, 1) * 2.0**-23
        r += c
    return d, s


@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
def test_wgrad(counts, N, K, kind):
    E, R = len(counts), sum(counts)
    M = R + 70
    gen = _gen(R * 3 + N + K)
    dC, A = _randn(gen, M, N), _randn(gen, M, K)
    dC[R:], A[R:] = float("nan"), float("inf")  # rows of no expert
    dt = BF16 if kind == "bf16" else torch.float32
    out = Guarded((E, N, K), dt, fill=0x7B)
    if kind == "add":
        out.t.copy_(_randn(gen, E, N, K, dtype=torch.float32, std=3.0))
    old = out.t.double()
    ws = _ws()
    moe.moe_grouped_gemm_wgrad(dC, A, _offsets(counts), M, E, N, K,
                               moe.MOE_GRAD_BF16 if kind == "bf16" else moe.MOE_GRAD_F32, kind == "add",
                               out.t, ws=ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0 and out.intact()
    d, eps = weights64(dC[:R], A[:R], counts)
    if kind == "add":
        d = d + old
        for e, c in enumerate(counts):
            if c == 0:
                assert torch.equal(out.t[e].double(), old[e])
    within(out.t, d, d.abs() * (2.0**-8 if kind == "bf16" else 2.0**-24) + eps, "dB")
    for e, c in enumerate(counts):
        if c == 0 and kind != "add":
            assert (out.t[e] == 0).all()


# few tiles and long sums: cut into parts where the workspace has room for them
@pytest.mark.parametrize("room", [256, 1 << 20, 1 << 24])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("counts,N,K", [([5], 4096, 128), ([0, 31, 2], 3200, 384), ([130, 1], 2048, 256)])
def test_dgrad_in_parts(counts, N, K, act, room):
    E, R, behind = len(counts), sum(counts), 9
    M = R + behind
    gen = _gen(N + room)
    dC, B = _randn(gen, M, N), _randn(gen, E, N, K, std=0.05)
    gated = ACTS[act] is not None
    gu = _randn(gen, M, 2 * K, std=2.0) if gated else None
    out = Guarded((M, 2 * K if gated else K), BF16, fill=0x7B)
    h = Guarded((M, K), BF16, fill=0x7B) if gated else None
    ws = Guarded((room,), torch.uint8, fill=0xFF)
    ws.t[:256] = 0
    before = out.t[R:].clone()
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets(counts), M, E, N, K, act, out.t, gu=gu, h=h.t if gated else None,
                               ws=ws.t)
    assert moe.moe_get_device_status(ws.t) == 0
    assert out.intact() and ws.intact() and torch.equal(out.t[R:].view(torch.int16), before.view(torch.int16))
    d, eps = rows64(dC[:R], B, counts)
    if not gated:
        within(out.t[:R], d, d.abs() * 2.0**-8 + eps, "dA")
        return
    g, u = gu[:R, :K].double(), gu[:R, K:].double()
    a, da = act64(ACTS[act], g)
    ref = torch.cat([d * u * da, d * a], 1)
    tol = ref.abs() * 2.0**-8 + torch.cat([eps * (u * da).abs(), eps * a.abs()], 1) + 2.0**-18 * torch.cat(
        [(1 + g.abs()) * (d * u).abs(), (1 + g.abs()) * (d * g).abs()], 1)
    within(out.t[:R], ref, tol, "gated gradients")
    assert h.intact()
    within(h.t[:R], a * u, (a * u).abs() * 2.0**-8 + 2.0**-18 * (1 + g.abs()) * (g * u).abs(), "h")


@pytest.mark.parametrize("room", [256, 1 << 20, 1 << 24])
@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
@pytest.mark.parametrize("counts,N,K", [([2600], 128, 128), ([4100, 0], 256, 384), ([2055, 3, 7000], 384, 128)])
def test_wgrad_in_parts(counts, N, K, kind, room):
    E, R = len(counts), sum(counts)
    M = R + 70
    gen = _gen(R + room)
    dC, A = _randn(gen, M, N), _randn(gen, M, K)
    dC[R:], A[R:] = float("nan"), float("inf")
    out = Guarded((E, N, K), BF16 if kind == "bf16" else torch.float32, fill=0x7B)
    if kind == "add":
        out.t.copy_(_randn(gen, E, N, K, dtype=torch.float32, std=3.0))
    old = out.t.double()
    ws = Guarded((room,), torch.uint8, fill=0xFF)
    ws.t[:256] = 0
    moe.moe_grouped_gemm_wgrad(dC, A, _offsets(counts), M, E, N, K,
                               moe.MOE_GRAD_BF16 if kind == "bf16" else moe.MOE_GRAD_F32, kind == "add", out.t, ws=ws.t)
    assert moe.moe_get_device_status(ws.t) == 0 and out.intact() and ws.intact()
    d, eps = weights64(dC[:R], A[:R], counts)
    d = d + old if kind == "add" else d
    within(out.t, d, d.abs() * (2.0**-8 if kind == "bf16" else 2.0**-24) + eps, "dB")


def test_inputs_and_outputs_inside_the_workspace():
    """Rows that live in the workspace (as a forward leaves them) are not overwritten by partial sums."""
    E, R, N, K = 1, 24, 4096, 128
    gen = _gen(21)
    dC, B = _randn(gen, R, N), _randn(gen, E, N, K, std=0.05)
    ws = _ws(1 << 24)
    inside = ws[1024:1024 + R * N * 2].view(BF16).view(R, N)
    inside.copy_(dC)
    want, got = (torch.empty(R, K, dtype=BF16, device="cuda") for _ in range(2))
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets([R]), R, E, N, K, 0, want, ws=_ws(256))
    moe.moe_grouped_gemm_dgrad(inside, B, _offsets([R]), R, E, N, K, 0, got, ws=ws)
    assert torch.equal(inside, dC) and torch.equal(want, got)
    out = ws[1 << 22:(1 << 22) + R * K * 2].view(BF16).view(R, K)
    moe.moe_grouped_gemm_dgrad(dC, B, _offsets([R]), R, E, N, K, 0, out, ws=ws)
    assert torch.equal(out, want)
    R, N = 4000, 128
    dC, A = _randn(gen, R, N), _randn(gen, R, K)
    inside = ws[1024:1024 + R * N * 2].view(BF16).view(R, N)
    inside.copy_(dC)
    want, got = (torch.empty(1, N, K, device="cuda") for _ in range(2))
    moe.moe_grouped_gemm_wgrad(dC, A, _offsets([R]), R, 1, N, K, moe.MOE_GRAD_F32, 0, want, ws=_ws(256))
    moe.moe_grouped_gemm_wgrad(inside, A, _offsets([R]), R, 1, N, K, moe.MOE_GRAD_F32, 0, got, ws=ws)
    assert torch.equal(inside, dC) and torch.equal(want, got)


def test_wgrad_long_sums_stay_precise():
    """16384 rows of one expert: the fp32 sum stays within 1e-5 of the result's norm."""
    R, N, K = 16384 + 13, 256, 256
    gen = _gen(5)
    dC, A = _randn(gen, R, N), _randn(gen, R, K)
    out = torch.empty(1, N, K, device="cuda")
    moe.moe_grouped_gemm_wgrad(dC, A, _offsets([R]), R, 1, N, K, moe.MOE_GRAD_F32, 0, out, ws=_ws())
    ref = dC.double().T @ A.double()
    assert ((out[0].double() - ref).norm() / ref.norm()).item() < 1e-5
    # all of one sign: the running sum grows to its end
    dC, A = dC.abs(), A.abs()
    moe.moe_grouped_gemm_wgrad(dC, A, _offsets([R]), R, 1, N, K, moe.MOE_GRAD_F32, 0, out, ws=_ws())
    ref = dC.double().T @ A.double()
    assert ((out[0].double() - ref).norm() / ref.norm()).item() < 1e-5


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_experts_nan_stays_with_it(bad):
    counts = [70, 0, 21, 130, 5]
    E, R, N, K = len(counts), sum(counts), 256, 384
    gen = _gen(11)
    dC, A, B = _randn(gen, R, N), _randn(gen, R, K), _randn(gen, E, N, K)
    off = _offsets(counts)
    edges = off.tolist()

    def both():
        dA = torch.empty(R, K, dtype=BF16, device="cuda")
        dB = torch.empty(E, N, K, device="cuda")
        moe.moe_grouped_gemm_dgrad(dC, B, off, R, E, N, K, moe.MOE_EPILOGUE_NONE, dA, ws=_ws())
        moe.moe_grouped_gemm_wgrad(dC, A, off, R, E, N, K, moe.MOE_GRAD_F32, 0, dB, ws=_ws())
        return dA, dB

    clean = both()
    hit = 3
    dC[edges[hit]:edges[hit + 1]] = bad
    A[edges[hit]:edges[hit + 1]] = bad
    dA, dB = both()
    rows = torch.ones(R, dtype=torch.bool, device="cuda")
    rows[edges[hit]:edges[hit + 1]] = False
    assert torch.equal(dA[rows], clean[0][rows])
    for e in range(E):
        if e != hit:
            assert torch.equal(dB[e], clean[1][e]), e
    assert not torch.isfinite(dB[hit]).any() and not torch.isfinite(dA[~rows]).any()


def test_offsets_out_of_range_write_nothing_else():
    """Offsets past M_total (and below zero) are clamped."""
    E, M, N, K = 3, 40, 128, 128
    gen = _gen(2)
    dC, A, B = _randn(gen, M, N), _randn(gen, M, K), _randn(gen, E, N, K)
    off = torch.tensor([-9, 30, 25, 1000], dtype=torch.int32, device="cuda")  # rows [0, 30), none, [25, 40)
    dA = Guarded((M, K), BF16, fill=0x7B)
    dB = Guarded((E, N, K), torch.float32, fill=0x7B)
    moe.moe_grouped_gemm_wgrad(dC, A, off, M, E, N, K, moe.MOE_GRAD_F32, 0, dB.t, ws=_ws())
    moe.moe_grouped_gemm_dgrad(dC, B, off, M, E, N, K, moe.MOE_EPILOGUE_NONE, dA.t, ws=_ws())
    torch.cuda.synchronize()
    assert dA.intact() and dB.intact()
    for e, (lo, hi) in enumerate([(0, 30), (30, 30), (25, 40)]):
        d, s = weights64(dC[lo:hi], A[lo:hi], [hi - lo])
        within(dB.t[e:e + 1], d, d.abs() * 2.0**-24 + s, "dB")


def test_binding_refuses_strided_tensors():
    dC, B, dA = (torch.zeros(128, 256, dtype=BF16, device="cuda") for _ in range(3))
    for kw in (dict(dC=dC.t()), dict(B=B[:, ::2]), dict(dA=dA.t())):
        a = dict(dC=dC, B=B, offsets=_offsets([128]), M_total=128, E=1, N=128, K=128, ep=0, dA=dA, ws=_ws(256)) | kw
        with pytest.raises(moe.MoeError, match="dense"):
            moe.moe_grouped_gemm_dgrad(**a)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,H,k", [(1, 128, 1), (1, 128, 2), (3, 256, 3), (16, 4096, 2), (33, 1152, 4), (7, 7168, 8),
                                   (5, 384, 9), (64, 128, 16), (300, 640, 6)])
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_backward(T, H, k, in_place):
    gen = _gen(T + H + k)
    R = T * k
    dout, y = _randn(gen, T, H), _randn(gen, R, H)
    w = torch.rand(T, k, generator=gen, device="cuda") - 0.2
    inv = torch.randperm(R, generator=gen, device="cuda").to(torch.int32).view(T, k)
    dy = Guarded((R, H), BF16, fill=0x7B)
    dw = Guarded((T, k), torch.float32, fill=0x7B)
    yin = y
    if in_place:
        dy.t.copy_(y)
        yin = dy.t
    ws = _ws(256)
    moe.moe_combine_backward(dout, yin, w, inv, (T, H, 128, 16, k), dy.t, dw.t, ws=ws)
    torch.cuda.synchronize()
    assert dy.intact() and dw.intact() and moe.moe_get_device_status(ws) == 0
    i = inv.long()
    ref = torch.empty(R, H, dtype=torch.float64, device="cuda")
    ref[i.view(-1)] = (w.double()[..., None] * dout.double()[:, None]).view(R, H)
    within(dy.t, ref, ref.abs() * (2.0**-8 + 2.0**-23), "dy")
    prod = dout.double()[:, None] * y.double()[i]
    within(dw.t, prod.sum(-1), prod.abs().sum(-1) * H * 2.0**-24, "dw")


def test_combine_backward_records_a_bad_index():
    T, H, k = 4, 128, 2
    gen = _gen(1)
    dout, y = _randn(gen, T, H), _randn(gen, T * k, H)
    w = torch.rand(T, k, generator=gen, device="cuda")
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    inv[1, 0], inv[2, 1] = T * k, -1
    dy = Guarded((T * k, H), BF16, fill=0)
    dw = torch.full((T, k), 7.0, device="cuda")
    ws = _ws(256)
    moe.moe_combine_backward(dout, y, w, inv, (T, H, 128, 4, k), dy.t, dw, ws=ws)
    assert moe.moe_get_device_status(ws) == (moe.MOE_ERR_INVALID_ARG << 8) | 6
    assert dy.intact() and dw[1, 0] == 0 and dw[2, 1] == 0
    assert (dy.t[2] == 0).all() and (dy.t[5] == 0).all() and (dy.t[3] != 0).any()
    moe.moe_combine_backward(dout, y, w, inv, (T, H, 128, 4, k), dy.t, dw)  # without a status word


# ------------------------------------------------------------ orthogonalize
def newton64(G, steps, coeffs=COEFFS, eps=1e-7, scale=1.0):
    a, b, c = coeffs
    out = []
    for g in G.double():
        x = g / (g.norm() + eps)
        for _ in range(steps):
            if x.shape[0] <= x.shape[1]:
                s = x @ x.T
                x = a * x + (b * s + c * s @ s) @ x
            else:
                s = x.T @ x
                x = a * x + x @ (b * s + c * s @ s)
        out.append(x * scale)
    return torch.stack(out)


def orth(G, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0, ws=None):
    nb, m, n = G.shape
    out = Guarded((nb, m, n), BF16, fill=0x7B)
    if ws is None:
        ws = Guarded((moe.moe_orthogonalize_workspace_size(nb, m, n),), torch.uint8, fill=0xFF)
        ws.t[:256] = 0
    guard, ws = (ws, ws.t) if isinstance(ws, Guarded) else (None, ws)
    moe.moe_orthogonalize(G, nb, m, n, moe.MOE_GRAD_F32 if G.dtype == torch.float32 else moe.MOE_GRAD_BF16, steps,
                          coeffs, eps, scale, out.t, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0 and out.intact() and (guard is None or guard.intact())
    return out.t


def check_orth(got, ref, steps):
    assert torch.isfinite(got).all()
    for i in range(ref.shape[0]):
        norm = ref[i].norm()
        if norm == 0:
            assert (got[i] == 0).all()
            continue
        err = ((got[i].double() - ref[i]).norm() / norm).item()
        assert err <= 2.0**-8 + steps * 3 * 2.0**-11, (i, err)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("nb,rows,cols", [(1, 1, 1), (1, 1, 7), (2, 9, 1), (2, 5, 3), (1, 64, 64), (3, 65, 130),
                                          (2, 130, 65), (2, 128, 384), (2, 384, 128), (1, 257, 1000), (1, 1000, 257),
                                          (1, 320, 320), (5, 40, 72), (1, 2000, 24), (2, 513, 769), (3, 4, 4),
                                          (2, 7, 1024), (2, 1023, 8), (1, 9, 1500), (2, 3000, 5), (3, 6, 9001), (150, 2, 3)])
def test_orthogonalize(nb, rows, cols, dtype):
    G = _randn(_gen(rows * 3 + cols), nb, rows, cols, dtype=dtype)
    check_orth(orth(G), newton64(G, 5), 5)


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("nb,p,q", [(2, 9, 9), (1, 16, 64), (1, 31, 65), (1, 32, 511), (2, 33, 128), (1, 34, 1000),
                                    (1, 60, 61), (2, 64, 513), (1, 65, 1025), (1, 72, 192), (3, 97, 97), (1, 104, 1536),
                                    (1, 127, 2047), (1, 128, 2048), (1, 128, 2049), (2, 10, 3000), (1, 128, 4096),
                                    (1, 77, 4097), (10, 64, 2500), (1, 129, 512), (40, 20, 300),
                                    (30, 128, 700), (160, 24, 257), (20, 100, 2000)])
def test_orthogonalize_short_sides(nb, p, q, tall):
    """Every size of cluster, rows that end inside a warp's or a CTA's share, slices that end past the matrix."""
    G = _randn(_gen(p * 7 + q), nb, *((q, p) if tall else (p, q)), dtype=torch.float32 if q % 2 else BF16)
    check_orth(orth(G), newton64(G, 5), 5)


@pytest.mark.parametrize("shape", [(1, 100, 1800), (3, 640, 128), (1, 17, 600)])
def test_orthogonalize_short_sides_of_low_rank(shape):
    gen = _gen(17)
    nb, m, n = shape
    G = _randn(gen, nb, m, 3, dtype=torch.float32) @ _randn(gen, nb, 3, n, dtype=torch.float32)
    check_orth(orth(G), newton64(G, 5), 5)


def test_orthogonalize_short_sides_beside_other_kernels():
    """Clusters that hold their SMs whole, on two streams with pairs of SMs that do likewise; captured, too."""
    R, N, K = 3000, 512, 512
    gen = _gen(23)
    dC, A, off = _randn(gen, R, N), _randn(gen, R, K), _offsets([R])
    G, H = _randn(gen, 20, 96, 1000, dtype=torch.float32), _randn(gen, 2, 700, 128, dtype=torch.float32)

    def run(spaces):
        dB = torch.empty(1, N, K, device="cuda")
        out = [torch.empty(t.shape, dtype=BF16, device="cuda") for t in (G, H)]
        for _ in range(3):
            for t, o, w in zip((G, H), out, spaces[1:]):
                moe.moe_orthogonalize(t, *t.shape, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, o, w)
            moe.moe_grouped_gemm_wgrad(dC, A, off, R, 1, N, K, moe.MOE_GRAD_F32, 0, dB, ws=spaces[0])
        return [dB, *out]

    def spaces():
        return [_ws(1 << 23), *(_ws(moe.moe_orthogonalize_workspace_size(*t.shape)) for t in (G, H))]

    want = [t.clone() for t in run(spaces())]
    for t, ref in zip((G, H), want[1:]):
        check_orth(ref, newton64(t, 5), 5)
    two, streams, got = [spaces(), spaces()], [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(4):
        for s, sp in zip(streams, two):
            with torch.cuda.stream(s):
                got.append(run(sp))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(run(two[0]))
    for _ in range(2):
        for t in got[-1]:
            t.fill_(7)
        graph.replay()
    torch.cuda.synchronize()
    for outs in got:
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
    assert all(moe.moe_get_device_status(w) == 0 for sp in two for w in sp)


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("shape", [(2, 96, 200), (2, 200, 96)])
def test_orthogonalize_steps_and_scale(shape, steps):
    G = _randn(_gen(steps), *shape, dtype=torch.float32, std=1e-3)
    check_orth(orth(G, steps=steps, scale=-0.25), newton64(G, steps, scale=-0.25), steps)


@pytest.mark.parametrize("rank", [1, 4, 20])
@pytest.mark.parametrize("shape", [(1, 192, 448), (1, 448, 192)])
def test_orthogonalize_low_rank(shape, rank):
    """The directions outside the matrix's range stay there: roundings of X must not be multiplied up."""
    gen = _gen(rank)
    nb, m, n = shape
    G = _randn(gen, nb, m, rank, dtype=torch.float32) @ _randn(gen, nb, rank, n, dtype=torch.float32)
    check_orth(orth(G), newton64(G, 5), 5)


@pytest.mark.parametrize("cols", [72, 71])
@pytest.mark.parametrize("power", [-30, 0, 36, 37.9])
def test_orthogonalize_any_magnitude(power, cols):
    """Squares of large entries leave the fp32 range, and so may the norm and its inverse."""
    G = (_randn(_gen(9), 2, 400, cols, dtype=torch.float32).clamp(-4, 4).double() * 10.0**power).float()
    check_orth(orth(G, eps=0.0), newton64(G, 5, eps=0.0), 5)


def test_orthogonalize_cubic_converges_to_the_polar_factor():
    G = _randn(_gen(4), 1, 64, 256, dtype=torch.float32)
    out = orth(G, steps=20, coeffs=(1.5, -0.5, 0.0)).double()
    u, _, vt = torch.linalg.svd(G.double(), full_matrices=False)
    err = ((out - u @ vt).norm() / (u @ vt).norm()).item()
    assert err <= 2.0**-8 + 20 * 3 * 2.0**-11, err


def test_orthogonalize_zero_and_nan_matrices_stay_apart():
    G = _randn(_gen(6), 5, 70, 90, dtype=torch.float32)
    G[1] = 0
    clean = orth(G).clone()
    assert (clean[1] == 0).all()
    G[3, 2, 5] = float("nan")
    G[4, 0, 0] = float("inf")
    out = torch.empty(5, 70, 90, dtype=BF16, device="cuda")
    ws = _ws(moe.moe_orthogonalize_workspace_size(5, 70, 90))
    moe.moe_orthogonalize(G, 5, 70, 90, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, out, ws)
    assert torch.equal(out[:3], clean[:3])
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).all()


@pytest.mark.parametrize("shape", [(7, 72, 136), (7, 137, 61), (7, 72, 2500), (7, 3100, 260)])
def test_orthogonalize_in_passes_equals_at_once(shape):
    """A workspace that holds some of the stack: the same bits."""
    G = _randn(_gen(8), *shape, dtype=torch.float32)
    whole = orth(G)
    for hold in (1, 2, 3, 6):
        n = moe.moe_orthogonalize_workspace_size(hold, *shape[1:])
        assert torch.equal(orth(G, ws=_ws(n)), whole), hold


# ---------------------------------------------------- together, as they are used
def _layer(T, H, I, E, k, seed):
    gen = _gen(seed)
    x, wr = _randn(gen, T, H), _randn(gen, H, E, std=0.1)
    w13, w2 = _randn(gen, E, 2 * I, H, std=0.05), _randn(gen, E, H, I, std=0.05)
    return x, wr, w13, w2, _randn(gen, T, H)


def _experts_step(d, x, ids, w, w13, w2, dout, ws, act=moe.MOE_EPILOGUE_SWIGLU):
    """Forward pieces, then the gradients of everything from the combine down to x."""
    T, H, I, E, k = d
    R = T * k
    new = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    off, pt, ip = new(E + 1, dt=torch.int32), new(R, dt=torch.int32), new(T, k, dt=torch.int32)
    xp, gu, h, y, out = new(R, H), new(R, 2 * I), new(R, I), new(R, H), new(T, H)
    moe.moe_permute(ids, d, off, pt, ip, x, xp, ws)
    moe.moe_grouped_gemm(xp, w13, off, R, E, 2 * I, H, moe.MOE_DTYPE_BF16, moe.MOE_EPILOGUE_NONE, gu, ws=ws)
    moe.moe_grouped_gemm(xp, w13, off, R, E, I, H, moe.MOE_DTYPE_BF16, act, h, ws=ws)
    moe.moe_grouped_gemm(h, w2, off, R, E, H, I, moe.MOE_DTYPE_BF16, moe.MOE_EPILOGUE_NONE, y, ws=ws)
    moe.moe_combine(y, w, ip, d, out)
    dy, dw = new(R, H), new(T, k, dt=torch.float32)
    moe.moe_combine_backward(dout, y, w, ip, d, dy, dw, ws=ws)
    dgu, h2 = new(R, 2 * I), new(R, I)
    moe.moe_grouped_gemm_dgrad(dy, w2, off, R, E, H, I, act, dgu, gu=gu, h=h2, ws=ws)
    dw2 = new(E, H, I, dt=torch.float32)
    moe.moe_grouped_gemm_wgrad(dy, h2, off, R, E, H, I, moe.MOE_GRAD_F32, 0, dw2, ws=ws)
    dxp, dx = new(R, H), new(T, H)
    moe.moe_grouped_gemm_dgrad(dgu, w13, off, R, E, 2 * I, H, moe.MOE_EPILOGUE_NONE, dxp, ws=ws)
    dw13 = new(E, 2 * I, H, dt=torch.float32)
    moe.moe_grouped_gemm_wgrad(dgu, xp, off, R, E, 2 * I, H, moe.MOE_GRAD_F32, 0, dw13, ws=ws)
    ones = torch.ones(T, k, device="cuda")
    moe.moe_combine(dxp, ones, ip, d, dx)
    return dict(out=out, dx=dx, dw=dw, dw13=dw13, dw2=dw2)


def _layer64(x, ids, w, w13, w2, act):
    """out[t] = sum_j w_j W2_e (act(Wg_e x) * (Wu_e x)) in fp64, dense over the experts, differentiable."""
    out = 0
    I = w2.shape[2]
    for e in range(w13.shape[0]):
        we = (w * (ids == e)).sum(1, keepdim=True)
        gu = x @ w13[e].T
        a, _ = act64(act, gu[:, :I])
        out = out + we * ((a * gu[:, I:]) @ w2[e].T)
    return out


@pytest.mark.parametrize("act", [moe.MOE_EPILOGUE_SWIGLU, moe.MOE_EPILOGUE_GEGLU, moe.MOE_EPILOGUE_REGLU])
@pytest.mark.parametrize("d", [(1, 128, 128, 4, 2), (64, 128, 256, 8, 2), (200, 384, 256, 16, 3)])
def test_layer_gradients(d, act):
    """The whole chain against autograd of the fp64 layer and against differences of its loss.

    Every intermediate is rounded to bf16 once (gu, h, y, dy, dgu, dx per slot): at most six roundings of half a
    step, 2^-8 each, lie between the inputs and any gradient, so each gradient's norm is off by 6 2^-8 at most."""
    T, H, I, E, k = d
    x, wr, w13, w2, dout = _layer(*d, seed=T)
    ws = _ws(moe.moe_workspace_size(d))
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    moe.moe_route_topk(x, wr, None, d, torch.empty(T, E, device="cuda"), ids, w)
    got = _experts_step(d, x, ids, w, w13, w2, dout, ws, act)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0
    P = dict(dx=x, dw=w, dw13=w13, dw2=w2)
    P = {n: p.double().requires_grad_(True) for n, p in P.items()}
    loss = lambda x, w, w13, w2: (_layer64(x, ids, w, w13, w2, ACTS[act]) * dout.double()).sum()  # noqa: E731
    grads = torch.autograd.grad(loss(P["dx"], P["dw"], P["dw13"], P["dw2"]), list(P.values()))
    for (name, p), ref in zip(P.items(), grads):
        err = ((got[name].double() - ref).norm() / ref.norm()).item()
        assert err <= 6 * 2.0**-8, (name, err)
        # a difference of the loss along the computed gradient itself
        if act != moe.MOE_EPILOGUE_REGLU:  # (smooth)
            v = got[name].double() / got[name].double().norm()
            args = {n: q.detach() for n, q in P.items()}
            step = 1e-4 * p.detach().norm()
            hi, lo = args | {name: args[name] + step * v}, args | {name: args[name] - step * v}
            slope = (loss(hi["dx"], hi["dw"], hi["dw13"], hi["dw2"]) - loss(lo["dx"], lo["dw"], lo["dw13"], lo["dw2"])) / (2 * step)
            norm = got[name].double().norm()
            assert abs(slope.item() - norm.item()) <= 8 * 2.0**-8 * norm.item(), (name, slope.item(), norm.item())


def test_training_step_is_repeatable_and_captures():
    """Two runs give the same bits; a captured step replays on new inputs, also after other graphs' work."""
    d = (96, 256, 384, 8, 2)
    T, H, I, E, k = d
    x, wr, w13, w2, dout = _layer(*d, seed=1)
    ids = torch.stack([torch.randperm(E, generator=_gen(t), device="cuda")[:k] for t in range(T)]).to(torch.int32)
    w = torch.softmax(_randn(_gen(2), T, k, dtype=torch.float32), 1)
    ws = _ws(moe.moe_workspace_size(d))
    ows = _ws(moe.moe_orthogonalize_workspace_size(E, H, I))
    upd = torch.empty(E, H, I, dtype=BF16, device="cuda")

    def step():
        g = _experts_step(d, x, ids, w, w13, w2, dout, ws)
        moe.moe_orthogonalize(g["dw2"], E, H, I, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, upd, ows)
        return g | dict(upd=upd)

    first = {n: t.clone() for n, t in step().items()}
    again = step()
    for n in first:
        assert torch.equal(first[n], again[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(_randn(_gen(77), T, H))
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: t.clone() for n, t in held.items()}
    eager = step()
    for n in eager:
        assert torch.equal(replayed[n], eager[n]), n
    assert not torch.equal(replayed["dx"], first["dx"])


@pytest.mark.parametrize("ahead", ["nothing", "memset", "copy", "join"])
def test_captured_alone_and_behind_other_nodes(ahead):
    """Launches that may start early, as a graph's first node and behind nodes that are no kernels."""
    R, N, K = 2600, 128, 256
    gen = _gen(31)
    G, M = _randn(gen, 2, 300, 200, dtype=torch.float32), _randn(gen, 2, 5, 90, dtype=torch.float32)
    dC, A, B = _randn(gen, R, N), _randn(gen, R, K), _randn(gen, 1, N, K)
    src, off = G.clone(), _offsets([R])
    O, O2 = torch.empty(2, 300, 200, dtype=BF16, device="cuda"), torch.empty(2, 5, 90, dtype=BF16, device="cuda")
    dB, dA = torch.empty(1, N, K, device="cuda"), torch.empty(R, K, dtype=BF16, device="cuda")
    wss = [_ws(1 << 23), _ws(moe.moe_orthogonalize_workspace_size(2, 300, 200)),
           _ws(moe.moe_orthogonalize_workspace_size(2, 5, 90))]

    def work():
        moe.moe_orthogonalize(G, 2, 300, 200, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, O, wss[1])
        moe.moe_orthogonalize(M, 2, 5, 90, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, O2, wss[2])
        moe.moe_grouped_gemm_wgrad(dC, A, off, R, 1, N, K, moe.MOE_GRAD_F32, 0, dB, ws=wss[0])
        moe.moe_grouped_gemm_dgrad(dC, B, off, R, 1, N, K, 0, dA, ws=wss[0])

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (O, O2, dB, dA)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if ahead == "memset":
            moe.moe_clear_device_status(wss[1])
        elif ahead == "copy":
            G.copy_(src)
        elif ahead == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                G.copy_(src)
            dC.mul_(1.0)
            torch.cuda.current_stream().wait_stream(side)
        work()
    for _ in range(3):
        for t in (O, O2, dB, dA):
            t.fill_(7)
        if ahead in ("copy", "join"):
            G.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((O, O2, dB, dA), want):
            assert torch.equal(t, w)


def test_two_streams_with_a_workspace_each():
    counts = [100, 3, 0, 261]
    E, R, N, K = len(counts), sum(counts), 384, 512
    gen = _gen(12)
    dC, A, B, off = _randn(gen, R, N), _randn(gen, R, K), _randn(gen, E, N, K), _offsets(counts)
    G = _randn(gen, 3, 200, 168, dtype=torch.float32)

    def run(ws, ows):
        dA = torch.empty(R, K, dtype=BF16, device="cuda")
        dB = torch.empty(E, N, K, device="cuda")
        O = torch.empty(3, 200, 168, dtype=BF16, device="cuda")
        moe.moe_grouped_gemm_dgrad(dC, B, off, R, E, N, K, moe.MOE_EPILOGUE_NONE, dA, ws=ws)
        moe.moe_grouped_gemm_wgrad(dC, A, off, R, E, N, K, moe.MOE_GRAD_F32, 0, dB, ws=ws)
        moe.moe_orthogonalize(G, 3, 200, 168, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, O, ows)
        return dA, dB, O

    n = moe.moe_orthogonalize_workspace_size(3, 200, 168)
    want = run(_ws(), _ws(n))
    spaces = [(_ws(), _ws(n)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, sp in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(run(*sp))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
