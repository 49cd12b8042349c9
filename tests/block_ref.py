"""fp64 definitions of the dense block operators (include/moe_block.h), in plain torch."""
import torch

F64 = torch.float64


def act(kind, g, u):
    s = torch.sigmoid(g)
    if kind == "situ":
        return 4 * torch.tanh(g / 4) * s * 25 * torch.tanh(u / 25)
    return g * s * u


def act_grads(kind, g, u):
    s = torch.sigmoid(g)
    if kind == "situ":
        a, b = 4 * torch.tanh(g / 4) * s, 25 * torch.tanh(u / 25)
        return (s / torch.cosh(g / 4) ** 2 + a * (1 - s)) * b, a / torch.cosh(u / 25) ** 2
    return (s + g * s * (1 - s)) * u, g * s


def ffn(kind, x, wg, wu, wd):
    x, wg, wu, wd = (t.to(F64) for t in (x, wg, wu, wd))
    return act(kind, x @ wg.T, x @ wu.T) @ wd.T


def ffn_grads(kind, x, wg, wu, wd, dy):
    """(dx, dwg, dwu, dwd) and the g, u they use."""
    x, wg, wu, wd, dy = (t.to(F64) for t in (x, wg, wu, wd, dy))
    g, u = x @ wg.T, x @ wu.T
    dh = dy @ wd
    ag, au = act_grads(kind, g, u)
    dg, du = dh * ag, dh * au
    return (dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ act(kind, g, u)), (g, u)


def norm(r, y, gate, w_post, w_next, eps=(1e-6, 1e-6), alpha=1.0, beta=1.0, stored=None):
    """(r_out, x); stored: r_out as its type keeps it, which the second norm reads."""
    r = r.to(F64)
    if y is not None:
        n = y.to(F64)
        if w_post is not None:
            n = n * (n.square().mean(1, keepdim=True) + eps[0]).rsqrt() * w_post.to(F64)
        r = alpha * r + beta * (1.0 if gate is None else gate.to(F64)) * n
    z = r if stored is None else r + (stored.to(F64) - r).detach()
    x = None if w_next is None else z * (z.square().mean(1, keepdim=True) + eps[1]).rsqrt() * w_next.to(F64)
    return r, x


def adamw(p, g, m, v, t, lr, betas, eps, wd, clip=1.0):
    """New (p, m, v) of step t in fp64."""
    p, g, m, v = (a.to(F64) for a in (p, g, m, v))
    g = g * clip
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    p = p * (1 - lr * wd) - lr / (1 - betas[0] ** t) * m / (v.sqrt() / (1 - betas[1] ** t) ** 0.5 + eps)
    return p, m, v
