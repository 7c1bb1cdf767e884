"""fp64 restatement of the operators of include/moe_ops.h on the CPU, straight
from their definitions (test infrastructure; shares no code with the kernels).
Inputs are torch CPU tensors of any type; results are fp64 (indices int64)."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
INF = math.inf


# ------------------------------------------------------------------------------ routing
def _masked(logits):
    l = logits.to(F64)
    return torch.where(torch.isnan(l), torch.full_like(l, -INF), l)


def scores(logits, kind):
    """[T, E] scores; 0 where the logit is -inf or NaN; a +inf logit is the limit."""
    l = _masked(logits)
    if kind == "sigmoid":
        return torch.sigmoid(l)
    top = l.max(1, keepdim=True).values
    e = torch.where(torch.isinf(top), (l == top).to(F64) * (top > 0), torch.exp(l - torch.where(torch.isinf(top), 0.0, top)))
    z = e.sum(1, keepdim=True)
    return torch.where(z > 0, e / torch.where(z > 0, z, 1.0), 0.0)


def shares(l, score):
    """s_j / sum s_j' over the last axis of chosen logits (-inf: masked), through log s, which does not
    underflow where s does; 0 where all are masked."""
    ls = torch.nn.functional.logsigmoid(l) if score == "sigmoid" else l
    top = ls.max(-1, keepdim=True).values
    # (a +inf logit is the limit; log sigmoid has no +inf)
    e = torch.where(torch.isinf(top), (ls == top).to(F64) * (top > 0), torch.exp(ls - torch.where(torch.isinf(top), 0.0, top)))
    z = e.sum(-1, keepdim=True)
    return torch.where(z > 0, e / torch.where(z > 0, z, 1.0), 0.0)


def route(logits, bias, k, groups=1, keep=None, group_top=1, score="sigmoid", renorm=True, scale=1.0):
    """(idx, w), token by token with Python's sort: a key and an index decide."""
    l, s = _masked(logits), scores(logits, score)
    T, E = l.shape
    keep = groups if keep is None else keep
    size = E // groups
    b = None if bias is None else bias.to(F64)
    idx = torch.zeros(T, k, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=F64)
    for t in range(T):
        lt, st = l[t].tolist(), s[t].tolist()
        key = lt if b is None else [x + y for x, y in zip(st, b.tolist())]
        val = st if b is None else key
        key = [-INF if q == -INF or kk != kk else kk for q, kk in zip(lt, key)]
        val = [-INF if q == -INF or v != v else v for q, v in zip(lt, val)]
        allowed = range(E)
        if keep < groups:
            if b is None and group_top == 1:
                val = key
            rank = []
            for g in range(groups):
                best = sorted(val[g * size:(g + 1) * size], reverse=True)[:group_top]
                finite = [v for v in best if v != -INF]
                rank.append((-sum(finite) if finite else INF, g))
            chosen = sorted(g for _, g in sorted(rank)[:keep])
            allowed = [e for g in chosen for e in range(g * size, (g + 1) * size)]
        order = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        idx[t] = torch.tensor(order)
        w[t] = (shares(l[t][idx[t]], score) if renorm else s[t][idx[t]]) * scale
    return idx, w


def route_weights(l, idx, score, renorm, scale):
    """w as a differentiable function of finite fp64 logits with idx held fixed."""
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = s.gather(1, idx)
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


def route_backward(logits, idx, dw, score="sigmoid", renorm=True, scale=1.0):
    """dl from the formulas; masked experts get and give nothing."""
    s = scores(logits, score)
    c = s.gather(1, idx)
    ds = dw.to(F64) * scale
    ds = torch.where(_masked(logits).gather(1, idx) == -INF, torch.zeros_like(ds), ds)
    if renorm:
        # ds_j ds_j/dl_j with the sum of scores divided out; softmax scores: the other terms cancel
        p = shares(_masked(logits).gather(1, idx), score)
        d = p * (ds - (p * ds).sum(1, keepdim=True))
        return torch.zeros_like(s).scatter_add(1, idx, d * (1.0 - c) if score == "sigmoid" else d)
    full = torch.zeros_like(s).scatter_add(1, idx, ds)
    if score == "sigmoid":
        return full * s * (1.0 - s)
    return s * (full - (c * ds).sum(1, keepdim=True))


# ------------------------------------------------------------------------------ norms
def norm(x, gamma, beta, eps, kind="layer"):
    """(y, mean, rstd)"""
    x = x.to(F64)
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=F64)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(c.pow(2).mean(1) + eps)
    y = c * rstd[:, None]
    y = y if gamma is None else y * gamma.to(F64)
    return (y if beta is None else y + beta.to(F64)), mean, rstd


def norm_backward(dy, x, gamma, mean, rstd, kind="layer"):
    """(dx, dgamma, dbeta) from given statistics (mean None for RMS norm)."""
    dy, x, r = dy.to(F64), x.to(F64), rstd.to(F64)[:, None]
    xh = (x - mean.to(F64)[:, None]) * r if kind == "layer" else x * r
    g = dy if gamma is None else dy * gamma.to(F64)
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return dx * r, (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------------------ linear
def act(a, kind):
    if kind == "relu":
        return torch.where(a > 0, a, torch.zeros_like(a))
    if kind == "silu":
        return a * torch.sigmoid(a)  # (a / (1 + e^-a) has no gradient where e^-a overflows)
    if kind == "gelu":
        return 0.5 * a * (1.0 + torch.erf(a / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)))
    return a


def act_grad(a, kind):
    a = a.to(F64).detach().requires_grad_(True)
    return torch.autograd.grad(act(a, kind).sum(), a)[0]


def linear(x, weight, bias, residual, kind):
    """(pre, y)"""
    pre = x.to(F64) @ weight.to(F64).T
    pre = pre if bias is None else pre + bias.to(F64)
    y = act(pre, kind)
    return pre, (y if residual is None else y + residual.to(F64))


def linear_backward(dy, pre, x, weight, kind):
    """(dp, dx, dweight, dbias), dp unrounded"""
    dp = dy.to(F64) if kind == "none" else dy.to(F64) * act_grad(pre, kind)
    return dp, dp @ weight.to(F64), dp.T @ x.to(F64), dp.sum(0)


# ------------------------------------------------------------------------------ clipping
def clip(grads, max_norm, kind="l2"):
    """(norm, [g * factor]); a norm past fp32 is infinite, and nothing is scaled"""
    gs = [g.to(F64).reshape(-1) for g in grads]
    flat = torch.cat(gs) if gs else torch.zeros(0, dtype=F64)
    if kind == "l2":
        norm = float(flat.pow(2).sum().sqrt())
    else:
        norm = float("nan") if torch.isnan(flat).any() else float(flat.abs().max()) if flat.numel() else 0.0
    if not math.isfinite(float(torch.tensor(norm, dtype=F64).to(torch.float32))):
        return (norm if math.isnan(norm) else INF), gs
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g * c for g in gs]
