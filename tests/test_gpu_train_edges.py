"""The training operators at the edges of what they document, against the formulas
in 64 bits. Tolerances count roundings as in test_gpu_train.py."""
import math
import os
import subprocess
import sys

import pytest

import orth_numbers as on
from helpers import Guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_tcgen05_b200 as moe  # noqa: E402

BF16 = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------- gates that are no numbers
def act64(act, g):
    """The activation and its derivative; a NaN gate makes both NaN."""
    if act == moe.MOE_EPILOGUE_SWIGLU:
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if act == moe.MOE_EPILOGUE_GEGLU:
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    da = torch.where(g > 0, 1.0, 0.0).double()
    return torch.clamp(g, min=0), torch.where(torch.isnan(g), g, da)


@pytest.mark.parametrize("act", [moe.MOE_EPILOGUE_SWIGLU, moe.MOE_EPILOGUE_GEGLU, moe.MOE_EPILOGUE_REGLU])
@pytest.mark.parametrize("N,room", [(256, 256), (4096, 1 << 24)])  # one launch; the sum in parts, added by another
@pytest.mark.parametrize("R", [40, 5])
def test_gates_that_are_no_numbers(R, N, room, act):
    """NaN and Inf in a gate or an up value reach what the formulas say and nothing else."""
    K = 128
    gen = _gen(R + N + act)
    dC, B, gu = _randn(gen, R, N), _randn(gen, 1, N, K, std=0.05), _randn(gen, R, 2 * K)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")

    def run(gu):
        out = torch.zeros(R, 2 * K, dtype=BF16, device="cuda")
        h = torch.zeros(R, K, dtype=BF16, device="cuda")
        ws = _ws(room)
        moe.moe_grouped_gemm_dgrad(dC, B, off, R, 1, N, K, act, out, gu=gu, h=h, ws=ws)
        assert moe.moe_get_device_status(ws) == 0
        return torch.cat([out, h], 1).double()

    clean, bad = run(gu), gu.clone()
    values = [math.nan, math.inf, -math.inf]
    for i, v in enumerate(values):
        bad[1, 7 * i] = v  # gates
        bad[R - 1, K + 5 * i + 1] = v  # up values
    got = run(bad)
    d = dC.double() @ B[0].double()
    eps = (dC.double().abs() @ B[0].double().abs()) * N * 2.0**-23
    g, u = bad[:, :K].double(), bad[:, K:].double()
    a, da = act64(act, g)
    ref = torch.cat([d * u * da, d * a, a * u], 1)
    slack = 2.0**-18 * (1 + g.abs())
    tol = ref.abs() * 2.0**-8 + torch.cat([eps * (u * da).abs() + slack * (d * u).abs(),
                                           eps * a.abs() + slack * (d * g).abs(), slack * (g * u).abs()], 1)
    real = torch.isfinite(ref)
    assert ((got - ref).abs() <= tol)[real].all()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    rest = ~real & ~torch.isnan(ref)
    assert torch.equal(got[rest], ref[rest])  # infinities, with their signs
    assert torch.isnan(got[1, [0, K, 2 * K]]).all()
    same = torch.ones_like(real)
    same[[1, R - 1]] = False
    assert torch.equal(got[same], clean[same])


# ----------------------------------------------- updates of large stacks
COEFFS = (3.4445, -4.7750, 2.0315)


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


def orth(G, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0, hold=None):
    """hold: matrices that the workspace has room for."""
    nb, m, n = G.shape
    out = Guarded((nb, m, n), BF16, fill=0x7B)
    ws = Guarded((moe.moe_orthogonalize_workspace_size(hold or nb, m, n),), torch.uint8, fill=0xFF)
    ws.t[:256] = 0
    moe.moe_orthogonalize(G, nb, m, n, moe.MOE_GRAD_F32 if G.dtype == torch.float32 else moe.MOE_GRAD_BF16, steps,
                          coeffs, eps, scale, out.t, ws.t)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws.t) == 0 and out.intact() and ws.intact()
    return out.t


def errors(got, ref):
    """Each matrix's distance from the reference, of the reference's norm."""
    assert torch.isfinite(got).all()
    return ((got.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)).max().item()


def orth_tol(steps):
    """Three operands a step are rounded to fp16, the result to bf16."""
    return 2.0**-8 + steps * 3 * 2.0**-11


# more than 296 tiles of 128 x 128: tiles of pairs of SMs; A's sum whole, and (one matrix) in parts
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("shape", [(20, 520, 1000), (20, 1000, 520), (6, 700, 2001), (6, 2001, 700), (5, 1500, 1500),
                                   (40, 260, 1028), (40, 1028, 260), (7, 3100, 260), (1, 300, 30000), (1, 30001, 257),
                                   (2, 513, 12000)])
def test_orthogonalize_large_stacks(shape, dtype):
    G = _randn(_gen(sum(shape)), *shape, dtype=dtype)
    ref = newton64(G, 5)
    err = errors(orth(G), ref)
    assert err <= orth_tol(5), err
    if shape[0] > 1:
        err = errors(orth(G, hold=max(1, shape[0] // 3)), ref)
        assert err <= orth_tol(5), err


@pytest.mark.parametrize("steps", [1, 2, 3])
@pytest.mark.parametrize("shape", [(20, 520, 1000), (20, 1000, 520), (6, 700, 2001), (6, 2001, 700)])
def test_orthogonalize_large_stacks_steps_and_rank(shape, steps):
    nb, m, n = shape
    G = _randn(_gen(steps), *shape, dtype=torch.float32, std=1e-3)
    err = errors(orth(G, steps=steps, scale=-0.25), newton64(G, steps, scale=-0.25))
    assert err <= orth_tol(steps), err
    gen = _gen(steps + 50)
    G = _randn(gen, nb, m, 4 * steps, dtype=torch.float32) @ _randn(gen, nb, 4 * steps, n, dtype=torch.float32)
    err = errors(orth(G), newton64(G, 5))
    assert err <= orth_tol(5), err


# ------------------------------------------------ the numbers of an update
@pytest.mark.parametrize("rank", [None, 4])
@pytest.mark.parametrize("shape", on.SHAPES)
def test_orthogonalize_is_as_exact_as_its_roundings(shape, rank):
    """No further from the formula than its own roundings, done on the CPU; alone, and in a stack of large tiles."""
    G = on.matrix(shape, rank)
    ref = on.newton64(G, 5)
    tol = on.MARGIN * on.distance(on.rounded(G, 5), ref)
    for nb in (1, 60):
        out = orth(G.cuda().expand(nb, *shape).contiguous()).cpu()
        err = on.distance(out[0], ref)
        assert err <= tol, (nb, err, tol)
        assert torch.equal(out, out[:1].expand(nb, *shape))


@pytest.mark.parametrize("nb,rows,cols", [(1, 4, 7), (3, 7, 4), (1, 16, 16), (2, 16, 700), (2, 700, 16), (1, 64, 2048),
                                          (1, 4000, 64), (1, 256, 256), (1, 300, 256), (1, 256, 2000),
                                          (80, 256, 300), (80, 300, 256)])
def test_orthogonalize_gives_the_diagonals_rest_back(nb, rows, cols):
    coeffs, value = on.diagonal_case(min(rows, cols))
    G = torch.eye(rows, cols, device="cuda").expand(nb, rows, cols).contiguous()
    assert torch.equal(orth(G, steps=1, coeffs=coeffs, eps=0.0), (G * value).to(BF16))


# ------------------------------------------------ norms that eps is not small beside
FORMS = [(3, 6, 500), (2, 1300, 4), (3, 40, 72), (2, 700, 100), (1, 60, 4000), (2, 130, 260), (2, 301, 190),
         (20, 520, 700), (20, 700, 515)]  # narrow, short in clusters of 1 to 16, tiles of one SM, of pairs


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("steps", [1, 5, 12])
@pytest.mark.parametrize("shape", FORMS)
def test_orthogonalize_small_norms(shape, steps, dtype):
    """X starts near |G| / eps and is as exact there; matrices of one stack each at their own size."""
    nb, m, n = shape
    eps = 1e-7
    unit = _randn(_gen(m + n + steps), nb, m, n, dtype=torch.float32) / math.sqrt(m * n)
    for norms in ([1e-7, 3e-8, 1.0], [1e-10, 1e-7, 1e-13], [1e-15, 1e-2, 1e-6], [1e-20, 1e-30, 1e-9], [2e-36, 5e-8, 1e-7]):
        size = torch.tensor((norms * nb)[:nb], device="cuda", dtype=torch.float64)[:, None, None]
        G = (unit.double() * size).to(dtype)
        err = errors(orth(G, steps=steps, eps=eps), newton64(G, steps, eps=eps))
        assert err <= orth_tol(steps), (norms, err)


@pytest.mark.parametrize("coeffs,steps,eps", [((1.5, -0.5, 0.0), 20, 1e3), ((1.875, -1.25, 0.375), 30, 1e5),
                                              ((3.4445, -4.7750, 2.0315), 64, 1e20), ((1.0, 0.0, 0.0), 3, 40.0),
                                              ((-2.0, 1.0, 0.0), 9, 1e6), ((0.5, 0.25, 0.25), 4, 100.0)])
@pytest.mark.parametrize("shape", [(2, 4, 100), (2, 40, 72), (1, 300, 130), (2, 130, 260), (20, 520, 700)])
def test_orthogonalize_large_eps(shape, coeffs, steps, eps):
    G = _randn(_gen(steps), *shape, dtype=torch.float32)
    ref = newton64(G, steps, coeffs, eps)
    err = errors(orth(G, steps=steps, coeffs=coeffs, eps=eps), ref)
    assert err <= orth_tol(steps), err


@pytest.mark.parametrize("eps", [1e-44, 1e-40, 1e-30, 1.0])
@pytest.mark.parametrize("shape", FORMS)
def test_orthogonalize_zero_matrices(shape, eps):
    """Zeros for any eps above zero, one whose inverse is no fp32 number included; their neighbours stay."""
    nb, m, n = shape
    G = _randn(_gen(m), nb, m, n, dtype=torch.float32)
    G[0] = 0
    out = orth(G, eps=eps)
    assert (out[0] == 0).all()
    if nb > 1:
        assert errors(out[1:], newton64(G[1:], 5, eps=eps)) <= orth_tol(5)


# ---------------------------------------------- polynomials at the end of the range
@pytest.mark.parametrize("nb,p,q", [(1, 9, 9), (2, 40, 100), (1, 100, 2047), (1, 128, 4096), (1, 200, 4096), (1, 130, 16383),
                                    (1, 300, 1 << 16), (20, 520, 1000), (3, 256, 16384)])
@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize_up_to_its_range(nb, p, q, tall):
    """Results are right up to the documented |X|_2 and polynomial, on a matrix whose one direction is an axis (its
    square has no smaller elements) and on one of full rank."""
    most = 65504 / math.sqrt(q)
    axis = torch.zeros(nb, p, q, device="cuda")
    axis[:, p // 2, q // 3] = 3.0
    for G in (axis, _randn(_gen(q), nb, p, q, dtype=torch.float32)):
        G = G.transpose(1, 2).contiguous() if tall else G
        x = 0.999 * math.sqrt(most)  # |X|_2 after the first step, if it was 1
        for steps, coeffs in ((2, (x - 0.9, 0.9, 0.0)), (1, (1.0, 0.0, 0.999 * most)), (1, (1.0, -0.999 * most, 0.0))):
            err = errors(orth(G, steps=steps, coeffs=coeffs), newton64(G, steps, coeffs))
            assert err <= orth_tol(steps), (steps, coeffs, err)


@pytest.mark.parametrize("shape", [(7, 72, 136), (4, 130, 260), (3, 301, 190), (20, 520, 700), (20, 700, 515), (3, 5, 600)])
def test_orthogonalize_one_matrix_that_is_no_number(shape):
    """NaN and Inf in one matrix, at its end and its start, reach no other; all of it is NaN."""
    G = _randn(_gen(sum(shape)), *shape, dtype=torch.float32)
    clean = orth(G).clone()
    G[1, -1, -1], G[2, 0, 0] = math.nan, math.inf
    out = torch.empty(shape, dtype=BF16, device="cuda")
    ws = _ws(moe.moe_orthogonalize_workspace_size(*shape))
    moe.moe_orthogonalize(G, *shape, moe.MOE_GRAD_F32, 5, COEFFS, 1e-7, 1.0, out, ws)
    assert moe.moe_get_device_status(ws) == 0
    rest = [i for i in range(shape[0]) if i not in (1, 2)]
    assert torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()


# ------------------------------------------------ elements past 2^31
def test_row_gradient_past_32_bits():
    """Rows whose results start past 2^31 elements: the last expert's against the formula, the first's too."""
    E, N, K, R = 2, 128, 4096, 530_000  # dA: 2.17e9 elements, with the gate 4.3e9
    gen = _gen(91)
    dC, B = _randn(gen, R, N), _randn(gen, E, N, K, std=0.05)
    off = torch.tensor([0, 300_000, R], dtype=torch.int32, device="cuda")
    probe = torch.tensor([0, 1, 299_999, 300_000, 524_287, 524_288, 529_000, R - 1], device="cuda")
    owner = (probe >= 300_000).long()
    d = torch.einsum("rn,rnk->rk", dC[probe].double(), B[owner].double())
    eps = torch.einsum("rn,rnk->rk", dC[probe].double().abs(), B[owner].double().abs()) * N * 2.0**-23
    out, ws = torch.empty(R, K, dtype=BF16, device="cuda"), _ws(256)
    moe.moe_grouped_gemm_dgrad(dC, B, off, R, E, N, K, moe.MOE_EPILOGUE_NONE, out, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    assert ((out[probe].double() - d).abs() <= d.abs() * 2.0**-8 + eps).all()
    del out
    gu = torch.empty(R, 2 * K, dtype=BF16, device="cuda")
    gu[:, :K], gu[:, K:] = 1.5, -0.75
    out, h = torch.empty(R, 2 * K, dtype=BF16, device="cuda"), torch.empty(R, K, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_dgrad(dC, B, off, R, E, N, K, moe.MOE_EPILOGUE_REGLU, out, gu=gu, h=h, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    for got, f in ((out[probe, :K], -0.75), (out[probe, K:], 1.5)):
        assert ((got.double() - f * d).abs() <= (f * d).abs() * 2.0**-8 + abs(f) * eps).all()
    assert (h == -1.125).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
def test_weight_gradient_past_32_bits(kind):
    E, N, K, each = 40, 8192, 8192, 19  # 2.7e9 elements
    R = E * each
    gen = _gen(92)
    dC, A = _randn(gen, R, N), _randn(gen, R, K)
    off = (torch.arange(E + 1, device="cuda") * each).to(torch.int32)
    out = torch.ones(E, N, K, dtype=BF16 if kind == "bf16" else torch.float32, device="cuda")
    ws = _ws(256)
    moe.moe_grouped_gemm_wgrad(dC, A, off, R, E, N, K, moe.MOE_GRAD_BF16 if kind == "bf16" else moe.MOE_GRAD_F32,
                               kind == "add", out, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    for e in (0, 31, 32, E - 1):  # 2^31 elements end with the 32nd expert
        x, y = dC[e * each:(e + 1) * each].double(), A[e * each:(e + 1) * each].double()
        for rows in (slice(0, 64), slice(N - 64, N)):
            ref, tol = x[:, rows].T @ y, (x[:, rows].abs().T @ y.abs()) * each * 2.0**-23
            ref = ref + (kind == "add")
            assert ((out[e, rows].double() - ref).abs() <= ref.abs() * (2.0**-8 if kind == "bf16" else 2.0**-24) + tol).all()


def test_combine_gradient_past_32_bits():
    T, H, k = 40_000, 7168, 8  # 2.3e9 elements of y
    gen = _gen(93)
    R = T * k
    dout = _randn(gen, T, H)
    y = torch.empty(R, H, dtype=BF16, device="cuda")
    y.copy_(torch.arange(1, R + 1, device="cuda")[:, None].remainder(251).expand(R, H))
    w = torch.rand(T, k, generator=gen, device="cuda")
    inv = torch.randperm(R, generator=gen, device="cuda").to(torch.int32).view(T, k)
    dw, ws = torch.empty(T, k, device="cuda"), _ws(256)
    factor = y[inv.long().view(-1), 0].double().view(T, k)
    moe.moe_combine_backward(dout, y, w, inv, (T, H, 128, 8, k), y, dw, ws=ws)
    assert moe.moe_get_device_status(ws) == 0
    total, size = dout.double().sum(1, keepdim=True), dout.double().abs().sum(1, keepdim=True)
    assert ((dw.double() - factor * total).abs() <= factor * size * H * 2.0**-24).all()
    for t in (0, 1, T // 2, T - 1):
        ref = w[t, :, None].double() * dout[t].double()
        assert ((y[inv[t].long()].double() - ref).abs() <= ref.abs() * (2.0**-8 + 2.0**-23)).all()
    last = inv.view(-1).argmax()  # the row at the end of y
    ref = w.view(-1)[last].double() * dout[last // k].double()
    assert ((y[R - 1].double() - ref).abs() <= ref.abs() * (2.0**-8 + 2.0**-23)).all()


@pytest.mark.parametrize("nb,rows,cols,hold", [(70_000, 128, 256, 70_000), (9000, 512, 512, 9000), (9000, 512, 512, 3000),
                                               (70_000, 8, 4096, 20_000)])
def test_update_past_32_bits(nb, rows, cols, hold):
    """Stacks of more than 2^31 elements and of more matrices than a grid's second axis counts."""
    one = _randn(_gen(94), 7, rows, cols, dtype=torch.float32)
    G = torch.empty(nb, rows, cols, dtype=BF16, device="cuda")
    for i in range(7):
        G[i::7] = one[i].to(BF16)
    out = torch.empty_like(G)
    ws = _ws(moe.moe_orthogonalize_workspace_size(hold, rows, cols))
    moe.moe_orthogonalize(G, nb, rows, cols, moe.MOE_GRAD_BF16, 3, COEFFS, 1e-7, 1.0, out, ws)
    assert moe.moe_get_device_status(ws) == 0
    assert errors(out[:7], newton64(G[:7], 3)) <= orth_tol(3)
    for i in range(7):
        assert torch.equal(out[i::7], out[i].expand(len(range(i, nb, 7)), rows, cols))


# ------------------------------------------------------- the first call of a process
FIRST = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
import mixture_experts_layer_tcgen05_b200 as moe
import test_gpu_train_edges as t
G = t._randn(t._gen(5), *{shape}, dtype=torch.float32)
out = torch.empty({shape}, dtype=torch.bfloat16, device="cuda")
ws = t._ws(moe.moe_orthogonalize_workspace_size(*{shape}))
R, N, K = 3000, 256, 128
dC, A, B, gu = t._randn(t._gen(6), R, N), t._randn(t._gen(7), R, K), t._randn(t._gen(8), 1, N, K), t._randn(t._gen(9), R, 2 * K)
off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
dA, dB, gws = torch.empty(R, 2 * K, dtype=torch.bfloat16, device="cuda"), torch.empty(1, N, K, device="cuda"), t._ws(1 << 24)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def calls():
    moe.moe_orthogonalize(G, *{shape}, moe.MOE_GRAD_F32, 5, t.COEFFS, 1e-7, 1.0, out, ws)
    moe.moe_grouped_gemm_dgrad(dC, B, off, R, 1, N, K, moe.MOE_EPILOGUE_SWIGLU, dA, gu=gu, ws=gws)
    moe.moe_grouped_gemm_wgrad(dC, A, off, R, 1, N, K, moe.MOE_GRAD_F32, 0, dB, ws=gws)
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (out, dA, dB)]
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, dA, dB)))
assert moe.moe_get_device_status(ws) == 0 and moe.moe_get_device_status(gws) == 0
assert t.errors(out, t.newton64(G, 5)) <= t.orth_tol(5)
"""


@pytest.mark.parametrize("shape", [(2, 4, 3000), (2, 128, 512), (1, 128, 4096), (1, 300, 200), (20, 520, 700)])
def test_first_call_of_a_process_is_captured(shape):
    """Kernels' attributes and the occupancy that a rule asks for are set while a stream is being captured."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests, shape=shape)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("coeffs,steps,eps", [((0.5, 0.25, 0.0), 5, 1e5), ((1.0, 1e4, 1e8), 2, 1e6), ((2.0, -1e3, 0.0), 1, 1e5),
                                              ((1.0, -1e12, 0.0), 1, 1e9), ((1e20, 0.0, 0.0), 1, 1e20),
                                              ((-1e20, 1.0, 0.0), 2, 1e38)])
@pytest.mark.parametrize("shape", [(2, 4, 100), (2, 40, 72), (1, 300, 130), (2, 130, 260), (20, 520, 700), (20, 700, 515)])
def test_orthogonalize_small_x_under_large_coefficients(shape, coeffs, steps, eps):
    """A polynomial whose coefficients are large while b A + c A^2 is not, on an X that eps makes small."""
    G = _randn(_gen(steps), *shape, dtype=torch.float32)
    err = errors(orth(G, steps=steps, coeffs=coeffs, eps=eps), newton64(G, steps, coeffs, eps))
    assert err <= orth_tol(steps), err
