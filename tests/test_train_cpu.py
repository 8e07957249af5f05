"""The training entry points on the CPU: host-side validation refuses bad calls
before any launch (no pointer here is ever dereferenced), and the workspace
sizes follow the documented bound."""
import pytest

import mixture_experts_layer_tcgen05_b200 as moe

# 16-byte aligned addresses far apart, never dereferenced
P = [0x7F0000000000 + (i << 36) for i in range(12)]
COEFFS = (3.4445, -4.7750, 2.0315)


def refused(fn, status, msg):
    with pytest.raises(moe.MoeError) as ei:
        fn()
    assert ei.value.status == status and msg in str(ei.value), str(ei.value)


def dgrad(**kw):
    a = dict(dC=P[0], B=P[1], offsets=P[2], M_total=64, E=4, N=256, K=128, ep=moe.MOE_EPILOGUE_NONE,
             dA=P[3], gu=None, h=None, ws=P[4], ws_bytes=256, stream=0) | kw
    return lambda: moe.moe_grouped_gemm_dgrad(**a)


def wgrad(**kw):
    a = dict(dC=P[0], A=P[1], offsets=P[2], M_total=64, E=4, N=256, K=128, type=moe.MOE_GRAD_F32,
             accumulate=0, dB=P[3], ws=P[4], ws_bytes=256, stream=0) | kw
    return lambda: moe.moe_grouped_gemm_wgrad(**a)


def combine(**kw):
    a = dict(dout=P[0], y_perm=P[1], w=P[2], inv_perm=P[3], d=(16, 128, 128, 4, 2), dy_perm=P[4],
             dw=P[5], ws=None, stream=0) | kw
    return lambda: moe.moe_combine_backward(**a)


def orth(**kw):
    a = dict(g=P[0], nb=2, rows=100, cols=60, g_type=moe.MOE_GRAD_F32, steps=5, coeffs=COEFFS, eps=1e-7,
             scale=1.0, out=P[1], ws=P[2], ws_bytes=1 << 30, stream=0) | kw
    return lambda: moe.moe_orthogonalize(**a)


INV, WS, DEV = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_UNSUPPORTED_DEVICE


@pytest.mark.parametrize("call", [dgrad(), wgrad(), combine(), orth(), dgrad(
    ep=moe.MOE_EPILOGUE_GEGLU, gu=P[5], h=P[6]), combine(dy_perm=P[1]), wgrad(accumulate=1)])
def test_valid_calls_reach_the_device_check(call, monkeypatch):
    monkeypatch.setenv("MOE_FAKE_CC", "90")
    refused(call, DEV, "sm_100a")


@pytest.mark.parametrize("kw,msg", [
    (dict(M_total=0), "M_total"), (dict(E=0), "E must"), (dict(E=1025), "E must"),
    (dict(N=100), "multiples of 128"), (dict(K=0), "multiples of 128"),
    (dict(E=1024, N=1 << 21), "2^31"), (dict(K=(1 << 24) + 128), "2^24"),
    (dict(dC=None), "dC is NULL"), (dict(offsets=None), "expert_offsets is NULL"),
    (dict(ws=None), "ws is NULL"), (dict(dC=P[0] + 8), "aligned"),
])
def test_grouped_gradients_refuse_bad_arguments(kw, msg):
    refused(dgrad(**kw), INV, msg)
    refused(wgrad(**kw), INV, msg)


def test_dgrad_refusals():
    refused(dgrad(ep=4), INV, "epilogue")
    refused(dgrad(ep=moe.MOE_EPILOGUE_SWIGLU), INV, "gu is NULL")
    refused(dgrad(gu=P[5]), INV, "gated")
    refused(dgrad(h=P[5]), INV, "gated")
    refused(dgrad(B=None), INV, "B is NULL")
    refused(dgrad(dA=None), INV, "dA is NULL")
    refused(dgrad(ws_bytes=255), WS, "small")
    # outputs over inputs: dC's last bytes, the weights, the workspace, each other
    refused(dgrad(dA=P[0] + 64 * 256 * 2 - 16), INV, "overlaps dC")
    refused(dgrad(dA=P[1]), INV, "overlaps B")
    refused(dgrad(dA=P[4]), INV, "overlaps ws")
    g = dict(ep=moe.MOE_EPILOGUE_SWIGLU, gu=P[5], h=P[6])
    refused(dgrad(**g | dict(dA=P[5])), INV, "overlaps gu")
    refused(dgrad(**g | dict(h=P[5])), INV, "overlaps gu")
    refused(dgrad(**g | dict(h=P[3] + 64 * 128 * 2)), INV, "dA and h overlap")


def test_wgrad_refusals():
    refused(wgrad(type=2), INV, "type")
    refused(wgrad(type=moe.MOE_GRAD_BF16, accumulate=1), INV, "fp32")
    refused(wgrad(A=None), INV, "A is NULL")
    refused(wgrad(dB=None), INV, "dB is NULL")
    refused(wgrad(ws_bytes=0), WS, "small")
    refused(wgrad(dB=P[1]), INV, "overlaps")
    refused(wgrad(dB=P[4]), INV, "overlaps")


def test_combine_backward_refusals():
    for d, msg in (((0, 128, 128, 4, 2), "T must"), ((16, 100, 128, 4, 2), "H must"),
                   ((16, 128, 128, 4, 5), "k must"), ((16, 128, 128, 2000, 2), "E must")):
        refused(combine(d=d), INV, msg)
    for name in ("dout", "y_perm", "w", "inv_perm", "dy_perm", "dw"):
        refused(combine(**{name: None}), INV, "NULL")
        refused(combine(**{name: P[7] + 4}), INV, "aligned")
    refused(combine(dy_perm=P[1] + 256), INV, "without being it")
    refused(combine(dy_perm=P[0]), INV, "overlaps dout")
    refused(combine(dw=P[2]), INV, "overlaps topk_w")
    refused(combine(dw=P[4]), INV, "dw overlaps")


def test_orthogonalize_refusals():
    for kw, msg in ((dict(nb=0), "nb"), (dict(rows=0), "rows and cols"), (dict(cols=(1 << 20) + 1), "rows and cols"),
                    (dict(nb=1 << 20, rows=1 << 12), "2^31"), (dict(g_type=5), "type"), (dict(steps=0), "steps"),
                    (dict(steps=65), "steps"), (dict(coeffs=(float("nan"), 1.0, 1.0)), "finite"),
                    (dict(scale=float("inf")), "finite"), (dict(eps=-1e-7), "eps"), (dict(g=None), "g is NULL"),
                    (dict(out=None), "out is NULL"), (dict(ws=None), "ws is NULL"), (dict(out=P[0]), "overlap"),
                    (dict(out=P[2]), "overlap"), (dict(ws=P[0] + (1 << 20) - (1 << 30), ), "overlap")):
        refused(orth(**kw), INV, msg)
    one = moe.moe_orthogonalize_workspace_size(1, 100, 60)
    refused(orth(ws_bytes=one - 1), WS, "one matrix")


@pytest.mark.parametrize("nb,rows,cols", [(1, 1, 1), (1, 1, 4097), (3, 64, 64), (2, 65, 129), (8, 512, 128),
                                          (32, 7168, 2048), (1, 1 << 20, 1), (64, 127, 63)])
def test_orthogonalize_workspace_follows_its_bound(nb, rows, cols):
    n = moe.moe_orthogonalize_workspace_size(nb, rows, cols)
    p = min(rows, cols)
    assert 0 < n <= 65536 + nb * (12 * (rows + 127) * (cols + 127) + 8 * (p + 127) ** 2)
    # the state's two halves, the upper one twice, and two squares, all fp16
    assert n >= nb * (6 * rows * cols + 4 * p * p)
    assert moe.moe_orthogonalize_workspace_size(nb + 1, rows, cols) > n
    for bad in ((0, rows, cols), (nb, 0, cols), (nb, rows, (1 << 20) + 1)):
        assert moe.moe_orthogonalize_workspace_size(*bad) == 0


def test_binding_refuses_tensors_elsewhere():
    """A CPU tensor's address is no device pointer."""
    torch = pytest.importorskip("torch")
    t = torch.zeros(64, 256, dtype=torch.bfloat16)
    for call in (dgrad(dC=t), wgrad(A=t), combine(dout=t), orth(g=t)):
        refused(call, INV, "current CUDA device")
