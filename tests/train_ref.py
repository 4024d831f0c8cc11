"""Float64 definitions of the training operators (torch, any device)."""
import torch


def pairs_of_rows(pair_row):
    """Inverse of pair_row: the flat (token, choice) pair of every expert-major row."""
    inv = torch.empty_like(pair_row, dtype=torch.long)
    inv[pair_row.long()] = torch.arange(pair_row.numel(), device=pair_row.device)
    return inv


def swiglu(gu, w_row):
    """w_row [R, 1] * SiLU(g) * u, in the type of gu."""
    g, u = gu.chunk(2, dim=1)
    return w_row * g * torch.sigmoid(g) * u


def swiglu_grad(dh, gu, w_row):
    """dgu and the row sums sum_c dh SiLU(g) u."""
    g, u = gu.chunk(2, dim=1)
    s = torch.sigmoid(g)
    act = g * s
    return (torch.cat([w_row * dh * u * s * (1 + g * (1 - s)), w_row * dh * act], 1),
            (dh * act * u).sum(1))


def route_weights(logits, ids, router):
    """Routing weights of the selected experts as a function of the logits."""
    if router == "softmax":
        return torch.softmax(logits.gather(1, ids), 1)
    if router == "full_softmax":
        return torch.softmax(logits, 1).gather(1, ids)
    s = torch.sigmoid(logits.gather(1, ids))
    return s / s.sum(1, keepdim=True)


def route_grad(logits, ids, dw, router):
    w = route_weights(logits, ids, router)
    own = dw - (w * dw).sum(1, keepdim=True)
    if router == "full_softmax":
        p = torch.softmax(logits, 1)
        d = torch.zeros_like(p).scatter_(1, ids, dw)
        return p * (d - (w * dw).sum(1, keepdim=True))
    d = w * own
    if router == "sigmoid_bias":
        d = d * (1 - torch.sigmoid(logits.gather(1, ids)))
    return torch.zeros_like(logits).scatter_(1, ids, d)


def rstd(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def block_norm(y, residual, w_post, gate, w_pre, alpha, eps, post, pre):
    """(s, x); gate a tensor that broadcasts over [N, H], or 1; y None: no block."""
    s = alpha * residual
    if y is not None:
        z = y * rstd(y, eps) if post else y
        if post and w_post is not None:
            z = z * w_post
        s = s + gate * z
    if not pre:
        return s, None
    x = s * rstd(s, eps)
    return s, x * w_pre if w_pre is not None else x
