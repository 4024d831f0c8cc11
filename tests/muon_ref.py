"""The orthogonalised momentum from its definition in 64 bits, and the same with the
roundings that the operator's documentation names."""
import math

import torch

P0, P1, P2 = 3.4445, -4.7750, 2.0315


def momentum(g, b, beta, nesterov):
    """(u, b')."""
    g = g.double()
    if b is None:
        return g, None
    b = beta * b.double() + g
    return (g + beta * b if nesterov else b), b


def orthogonal(u, steps, eps, rounded=False):
    """X of one matrix u [M, N] (float64).  rounded: G, S without its diagonal and X as an
    operand in fp16, scaled as the operator scales them (G and S by 2^12, X by 2^p)."""
    tall = u.shape[0] > u.shape[1]
    x = u.T if tall else u
    x = x / (torch.linalg.vector_norm(x) + eps)
    half = math.sqrt(max(u.shape))
    p = 2.0 ** round(math.log2(half))

    def r(t, scale):
        return (t * scale).half().double() / scale if rounded else t

    for _ in range(steps):
        xr = r(x, p)
        g = r(xr @ xr.T, 4096.0)
        s = P1 * g + P2 * (g @ g)
        d = torch.diagonal(s).clone()
        x = (P0 + d)[:, None] * x + r(s - torch.diag(d), 4096.0) @ xr
    return x.T if tall else x
