"""The numbers of moe_orthogonalize on the CPU: the formula in 64 bits, and the same
steps with the roundings that the kernels choose (each of which can be done otherwise,
to see what a bound on the error tells apart)."""
import math

import torch

COEFFS = (3.4445, -4.7750, 2.0315)


def newton64(G, steps, coeffs=COEFFS, eps=1e-7):
    a, b, c = coeffs
    wide = G.shape[0] <= G.shape[1]
    x = G.double() if wide else G.double().T
    x = x / (x.norm() + eps)
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    return x if wide else x.T


def rounded(G, steps, coeffs=COEFFS, eps=1e-7, operands=torch.float16, rest=True):
    """The state as two fp16 halves, the products' operands its upper half, A and b A + c A^2 (times a power of two
    s) in `operands`, sums in fp32; rest: what rounding takes from the diagonal of the last is given back."""
    a, b, c = coeffs
    wide = G.shape[0] <= G.shape[1]
    s = 2.0 ** math.floor(math.log2(max(G.shape)) / 2)
    x = (G if wide else G.T).float()
    x = x * (s / (x.double().norm().item() + eps))
    for _ in range(steps):
        up = x.to(operands).float()
        x = up + ((x - up) * 2048).half().float() / 2048
        A = (up @ up.T / s).to(operands).float()
        exact = b * A + (c / s) * (A @ A)
        B = exact.to(operands).float()
        back = (exact.diag() - B.diag()) / s if rest else torch.zeros(len(B))
        x = (a + back)[:, None] * x + (B @ up) / s
    x = (x / s).bfloat16()
    return x if wide else x.T


def distance(x, ref):
    return ((x.double() - ref).norm() / ref.norm()).item()


# White matrices and matrices of rank 4, wide and tall. The sum of an update's errors is that of thousands of
# independent roundings, whose size the order of the fp32 sums does not change: a kernel that rounds as `rounded`
# does is as far from the formula, to a few per cent. MARGIN leaves 15; bf16 operands are off by 1.5 to 6 times as much.
SHAPES = [(64, 64), (96, 200), (128, 384), (17, 600), (384, 96), (320, 320), (257, 1000), (1000, 257), (513, 769)]
MARGIN = 1.15


def matrix(shape, rank, seed=0):
    gen = torch.Generator().manual_seed(seed + sum(shape))
    if rank:
        return torch.randn(shape[0], rank, generator=gen) @ torch.randn(rank, shape[1], generator=gen)
    return torch.randn(*shape, generator=gen)


def diagonal_case(p):
    """One step of p orthogonal rows (p a power of 4) whose result, 9 2^-13 / sqrt(p) of them, every rounding but
    that of the diagonal of B = -(1 - 9 2^-13) leaves as it is; fp16 has -(1 - 8 2^-13). Coefficients and result."""
    b = -p * (1 - 9 * 2.0**-13) - 2.0 / p  # B = b / p + 2 / p^2
    return (1.0, b, 2.0), 9 * 2.0**-13 / math.sqrt(p)
