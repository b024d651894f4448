"""Binary64 references (torch, CPU) of the norm, the gate and the few-row
NVFP4 products, written from their definitions."""
from __future__ import annotations

import torch

U = 2.0 ** -24       # half a step of binary32, relative
HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative


def f64(t):
    return t.detach().cpu().double()


# ------------------------------------------------------------------ norm

def norm(total, weight, eps):
    """(y, rstd) of rows `total`, unrounded."""
    rstd = (total.square().mean(1) + eps).rsqrt()
    return total * rstd[:, None] * weight, rstd


def norm_backward(dy, x, weight, rstd, d_sum=None):
    """(dx, dw, bound of dx's binary32 error, sum of dw's absolute terms)."""
    r = rstd[:, None]
    g, h = dy * weight, x * r
    m = (g * h).mean(1, keepdim=True)
    dx = r * (g - h * m)
    # The products and the difference: 4 roundings on each side; the mean: at
    # most 64 additions a thread, 8 to join the threads, 4 roundings a term.
    size = r * (4 * g.abs() + h.abs() * (4 * m.abs() + 76 * (g * h).abs().mean(1, keepdim=True)))
    if d_sum is not None:
        dx = dx + d_sum
        size = size + d_sum.abs() + dx.abs()
    return dx, (dy * h).sum(0), 1.01 * U * size, (dy * h).abs().sum(0)


# ------------------------------------------------------------------ gate

def gate(z, k, softmax, renorm, scale, mask=None, coef=0.0):
    """dict of ids, prob, counts, prob_sum, loss (and v, p) for binary64 z."""
    T, E = z.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu() != 0
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    turn = torch.arange(T * k).view(T, k) % E
    ids = torch.where(live[:, None], ids, turn)
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    v, p = shares(zz, softmax)
    prob = v.gather(1, ids)
    if renorm:
        s = prob.sum(1, keepdim=True)
        prob = torch.where(s > 0, prob / s, torch.zeros_like(prob))
    prob = prob * scale * live[:, None]
    hits = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, 1.0) * live[:, None]
    counts, prob_sum, n = hits.sum(0), (p * live[:, None]).sum(0), int(live.sum())
    loss = coef * E * (counts * prob_sum).sum() / (k * n * n) if n else torch.zeros(()).double()
    return dict(ids=ids, prob=prob, counts=counts, n=n, prob_sum=prob_sum, loss=loss, v=v, p=p,
                live=live)


def shares(z, softmax):
    """A row's scores v and its shares p; an all -inf row has none."""
    if softmax:
        top = z.amax(1, keepdim=True)
        v = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        s = v.sum(1, keepdim=True)
        v = torch.where(s > 0, v / s, torch.zeros_like(v))
        return v, v
    v = 1.0 / (1.0 + torch.exp(-z))
    s = v.sum(1, keepdim=True)
    return v, torch.where(s > 0, v / s, torch.zeros_like(v))


def gate_objective(z, ids, counts, n, softmax, renorm, scale, live, coef, d_prob, d_loss):
    """What the gate's gradient is the gradient of, the choice held fixed."""
    v, p = shares(z, softmax)
    prob = v.gather(1, ids)
    if renorm:
        prob = prob / prob.sum(1, keepdim=True)
    out = (prob * scale * live[:, None] * d_prob).sum()
    k, E = ids.shape[1], z.shape[1]
    if n:
        out = out + d_loss * coef * E * (counts * (p * live[:, None]).sum(0)).sum() / (k * n * n)
    return out


def gate_backward(z, ids, counts, n, softmax, renorm, scale, live, coef, d_prob, d_loss):
    """(d_z, the size of the terms each element is the sum of)."""
    T, E = z.shape
    k = ids.shape[1]
    v, p = shares(z, softmax)
    sel, d = v.gather(1, ids), d_prob * scale
    size = d.abs()
    if renorm:
        s = sel.sum(1, keepdim=True)
        size = (size + (size * sel).sum(1, keepdim=True) / s) / s
        d = (d - (d * sel).sum(1, keepdim=True) / s) / s
    u = torch.zeros_like(z).scatter_add_(1, ids, d)
    us = torch.zeros_like(z).scatter_add_(1, ids, size)
    h = d_loss * coef * E * counts / (k * n * n) if n else torch.zeros(E).double()
    hs = h.abs()
    if softmax:
        dz = p * (u + h - (p * (u + h)).sum(1, keepdim=True))
        size = p * (us + hs + (p * (us + hs)).sum(1, keepdim=True))
    else:
        s = v.sum(1, keepdim=True)
        w = v * (1 - v)
        dz = w * (u + (h - (p * h).sum(1, keepdim=True)) / s)
        # 1 - v keeps an absolute error of U, whatever is left of it
        size = (w + v) * (us + (hs + (p * hs).sum(1, keepdim=True)) / s)
    return dz * live[:, None], size * live[:, None]


# ------------------------------------------------------------------ NVFP4

_E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def e4m3(byte):
    b = byte.cpu().long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -v, v)


def nvfp4(q, sb):
    """q s_b of packed rows [.., K/2] and scales [.., K/16], without s_g."""
    q = q.cpu()
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    v = _E2M1[codes & 7] * torch.where(codes >= 8, -1.0, 1.0).double()
    return (v.unflatten(-1, (-1, 16)) * e4m3(sb)[..., None]).flatten(-2)


def gemv(x, ids, q, sb, sg, N, rps, div):
    """(y, sum of the absolute terms) [rows, N]; rows of ids outside give 0."""
    rows, K = ids.numel(), x.shape[1]
    G = q.numel() // (N * (K // 2))
    y = torch.zeros(rows, N, dtype=torch.float64)
    size = torch.zeros(rows, N, dtype=torch.float64)
    q, sb, sg, x = q.cpu().view(G, N, -1), sb.cpu().view(G, N, -1), f64(sg), f64(x)
    flat = ids.cpu().view(-1).tolist()
    for e in sorted(set(flat)):
        if not 0 <= e < G:
            continue
        w = nvfp4(q[e], sb[e]) * sg[(e * N + torch.arange(N)) // rps][:, None]
        mine = [r for r in range(rows) if flat[r] == e]
        xr = x[[r // div for r in mine]]
        y[mine] = xr @ w.t()
        size[mine] = xr.abs() @ w.abs().t()
    return y, size


def gemv_bound(size, K):
    """Binary32 error of a sum whose operands are exact: 32 products a matrix
    instruction, K / 128 (rounded up) instructions a wave, four waves joined, one multiply by
    the outer scale; each step at most a whole step of binary32 (2 U), which
    covers an accumulator that truncates."""
    return (-(-K // 128) + 32 + 4 + 1) * 2 * U * size


def random_nvfp4(g, rows, K, std=0.02):
    """Random packed codes and block scales as weights have them."""
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    sb = torch.randint(48, 127, (rows, K // 16), generator=g, dtype=torch.uint8)
    return q, sb
