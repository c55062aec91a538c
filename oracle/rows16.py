"""64-bit oracle of the 16-bit products and of the routing by scores (torch,
on whatever device the operands are): written from the formulas, with nothing
of the HIP path."""
from __future__ import annotations

import math

import torch

LOWEST = torch.finfo(torch.float32).min


def activation(v, name: str):
    if name == "none":
        return v
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.special.erfc(-v * math.sqrt(0.5))
    if name == "gelu_tanh":
        return v * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(name)


def product(x, w, bias=None):
    """x w^T + bias, and the sum of the magnitudes that it is made of."""
    a, b = x.double(), w.double().t().contiguous()
    v, mag = a @ b, a.abs() @ b.abs()
    if bias is not None:
        v, mag = v + bias.double(), mag + bias.double().abs()
    return v, mag


def dense(x, w, bias=None, act="none", residual=None):
    v, _ = product(x, w, bias)
    v = activation(v, act)
    return v if residual is None else v + residual.double()


def gated(x, w, bias=None, act="silu"):
    v, _ = product(x, w, bias)
    F = w.shape[0] // 2
    return activation(v[:, :F], act) * v[:, F:]


def router(logits, k, bias=None, score="softmax", groups=1, top_groups=None, group_score="top2", renormalise=True,
           scale=1.0):
    """Ids [T, k] and 64-bit weights [T, k], row by row as the rule reads:
    scores in 64 bits, rounded to fp32 for the ranking; the weights are made of
    the rounded scores."""
    l = logits.double()
    T, E = l.shape
    top_groups = groups if top_groups is None else top_groups
    shut = torch.isnan(l) | torch.isneginf(l)
    l = torch.where(shut, torch.full_like(l, -math.inf), l.clamp(max=-LOWEST))
    if score == "softmax":
        top = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
    else:
        p = torch.sigmoid(l)
    s = p.float()
    b = torch.zeros(E, device=l.device) if bias is None else bias
    shut = shut | torch.isnan(b) | torch.isneginf(b)
    c = torch.where(shut, torch.full_like(s, LOWEST), (s + torch.where(torch.isnan(b), torch.zeros_like(b), b)).clamp(LOWEST, -LOWEST))
    s = torch.where(shut, torch.zeros_like(s), s)
    if top_groups < groups:
        size = E // groups
        m = torch.sort(c.view(T, groups, size), dim=2, descending=True)[0]
        gs = m[:, :, 0]
        if group_score == "top2":
            gs = gs + torch.where(m[:, :, 1] > LOWEST, m[:, :, 1], torch.zeros_like(gs))
        order = torch.sort(gs, dim=1, descending=True, stable=True)[1]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=l.device)
        keep.scatter_(1, order[:, :top_groups], True)
        c = torch.where(keep.repeat_interleave(size, 1), c, torch.full_like(c, -math.inf))
    idx = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :k]
    w = s.gather(1, idx).double()
    if renormalise:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return idx.int(), w * scale
