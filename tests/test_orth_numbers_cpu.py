"""What the bounds on an orthogonalised update's error tell apart, on the CPU."""
import math

import pytest

torch = pytest.importorskip("torch")

import orth_numbers as on  # noqa: E402


@pytest.mark.parametrize("rank", [None, 4])
@pytest.mark.parametrize("shape", on.SHAPES)
def test_the_margin_tells_bf16_operands_apart(shape, rank):
    G = on.matrix(shape, rank)
    ref = on.newton64(G, 5)
    err = on.distance(on.rounded(G, 5), ref)
    # three operands of half a step each and step, and the result's half step, all in one direction
    assert err <= 2.0**-8 + 5 * 3 * 2.0**-11
    assert on.distance(on.rounded(G, 5, operands=torch.bfloat16), ref) > on.MARGIN * err
    if rank is None:
        assert on.distance(on.rounded(G, 5, rest=False), ref) > err


@pytest.mark.parametrize("p", [4, 16, 64, 256])
def test_the_diagonal_case_tells_a_lost_rest_apart(p):
    coeffs, value = on.diagonal_case(p)
    for c in coeffs:
        assert torch.tensor(c, dtype=torch.float32).item() == c  # what a C float holds
    G = torch.eye(p, p + 3)
    want = (G * value).bfloat16()
    assert math.isclose(want[0, 0].item(), value, rel_tol=0)
    assert (on.newton64(G, 1, coeffs, 0.0) - want.double()).abs().max() < 1e-15
    assert torch.equal(on.rounded(G, 1, coeffs, 0.0), want)
    assert on.distance(on.rounded(G, 1, coeffs, 0.0, rest=False), want.double()) > 0.1
