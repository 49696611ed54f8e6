"""Plain 64-bit forms of the scored route, the experts' products and the combine's gradients, for the
GPU tests (CPU tensors, straight from the formulas; shares nothing with the library)."""
import math

import torch


def scores(logits, func):
    z = logits.double()
    if func == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def route(logits, k, func, renorm, groups=1, top_groups=1, group_top=1, scale=1.0, bias=None):
    """(ids, gates, key) with ties to the lower index."""
    T, E = logits.shape
    s = scores(logits, func)
    key = s if bias is None else s + bias.double()
    sel = key
    if top_groups < groups:
        parts = key.reshape(T, groups, E // groups)
        best = torch.sort(parts, dim=2, descending=True).values[:, :, :group_top].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, order, True)
        keep = keep[:, :, None].expand_as(parts).reshape(T, E)
        # experts of other groups sort behind every kept one, -inf keys included
        first = torch.sort((~keep).int(), dim=1, stable=True).indices
        n = top_groups * (E // groups)
        cand = first[:, :n]
        sub = torch.sort(torch.gather(key, 1, cand), dim=1, descending=True, stable=True).indices
        ids = torch.gather(cand, 1, sub[:, :k])
    else:
        ids = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :k]
    return ids, gates_of(s, ids, renorm, scale), key


def gates_of(s, ids, renorm, scale):
    g = torch.gather(s, 1, ids)
    if renorm:
        total = g.sum(1, keepdim=True)
        g = torch.where(total > 0, g / total, torch.zeros_like(g))
    return g * scale


def act(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z / math.sqrt(2.0)))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "swiglu":
        F = z.shape[-1] // 2
        return z[..., :F] * torch.sigmoid(z[..., :F]) * z[..., F:]
    return z


def segments(counts, off, capacity, E):
    c = [min(int(v), capacity) if capacity else int(v) for v in counts]
    return [slice(int(off[e]), int(off[e]) + c[e]) for e in range(E)]


def matmul(x, w, segs, bias=None, name="none", residual=None):
    """(out, pre, mag): mag bounds the terms of each z (sum of |x||w| + |bias|)."""
    E, W, K = w.shape
    F = W // 2 if name == "swiglu" else W
    n = x.shape[0]
    out = torch.zeros(n, F, dtype=torch.float64)
    pre = torch.zeros(n, W, dtype=torch.float64)
    mag = torch.zeros(n, W, dtype=torch.float64)
    for e, r in enumerate(segs):
        if r.stop > r.start:
            xe, we = x[r].double(), w[e].double()
            z = xe @ we.T
            m = xe.abs() @ we.abs().T
            if bias is not None:
                z = z + bias[e].double()
                m = m + bias[e].double().abs()
            pre[r], mag[r] = z, m
            y = act(z, name)
            out[r] = y if residual is None else y + residual[r].double()
    return out, pre, mag


def act_grad(z, d, name):
    z = z.detach().clone().requires_grad_(True)
    y = act(z, name)
    return torch.autograd.grad(y, z, d)[0]


def matmul_grads(dy, x, w, pre, segs, name="none"):
    """grad_x, grad_w, grad_bias, grad_pre and the magnitudes of their terms, in 64 bits."""
    E, W, K = w.shape
    n = x.shape[0]
    gx, mx = torch.zeros(n, K, dtype=torch.float64), torch.zeros(n, K, dtype=torch.float64)
    gw, mw = torch.zeros(E, W, K, dtype=torch.float64), torch.zeros(E, W, K, dtype=torch.float64)
    gb, mb = torch.zeros(E, W, dtype=torch.float64), torch.zeros(E, W, dtype=torch.float64)
    gp = torch.zeros(n, W, dtype=torch.float64)
    for e, r in enumerate(segs):
        if r.stop > r.start:
            d = dy[r].double()
            if name != "none":
                d = act_grad(pre[r].double(), d, name)
            gp[r] = d
            gx[r], mx[r] = d @ w[e].double(), d.abs() @ w[e].double().abs()
            gw[e], mw[e] = d.T @ x[r].double(), d.abs().T @ x[r].double().abs()
            gb[e], mb[e] = d.sum(0), d.abs().sum(0)
    return gx, gw, gb, gp, mx, mw, mb
