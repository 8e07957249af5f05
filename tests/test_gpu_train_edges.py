"""The training operators at the edges of what they document, against the formulas
in 64 bits. Tolerances count roundings as in test_gpu_train.py."""
import math

import pytest

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
