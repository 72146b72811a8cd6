"""Plain 64-bit forms of the row operators (norm, routing of given logits, combine's
gradient, linear layer), for the tests: written from the formulas in include/moe.h."""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step
INF = math.inf


def norm(x, w, b, eps, kind):
    x = x.double()
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = (((x - mean) ** 2).mean(1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32))) ** -0.5
    w = torch.ones_like(x[0]) if w is None else w.double()
    b = torch.zeros_like(x[0]) if b is None else b.double()
    return (x - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]


def norm_backward(dy, x, w, mean, rstd, kind):
    dy, x, r = dy.double(), x.double(), rstd.double()[:, None]
    n = (x - mean.double()[:, None]) * r if kind == "layer" else x * r
    g = dy if w is None else dy * w.double()
    dx = g - n * (g * n).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return dx * r, (dy * n).sum(0), dy.sum(0)


def scores(l, fn):
    if fn == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    if fn == "sqrtsoftplus":
        return torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))
    top = l.max(1, keepdim=True)[0]
    e = torch.exp(l - torch.where(top == -INF, 0.0, top))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def route(cfg, logits, bias):
    """Experts and weights: by s', then by the logit, then by the index."""
    l = logits.double().cpu()
    T, E = l.shape
    k, G = cfg.num_experts_per_tok, cfg.n_group
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    bad = (torch.isnan(l) | (l == INF)).any(1) | (torch.isnan(b) | (b == INF)).any()
    s = scores(torch.where(bad[:, None], 0.0, l), cfg.score_fn)
    sel = torch.where((l == -INF) | (b == -INF) | bad[:, None], -INF, s + b).numpy()
    if G > 1:
        two = -np.sort(-sel.reshape(T, G, E // G), axis=2)[:, :, :2]
        value = two[:, :, 0] if two.shape[2] < 2 else \
            np.where(two[:, :, 1] == -INF, two[:, :, 0], two.sum(2))
        keep = np.argsort(-value, axis=1, kind="stable")[:, :cfg.topk_group]
        kept = np.zeros((T, G), bool)
        np.put_along_axis(kept, keep, True, 1)
        sel = np.where(np.repeat(kept, E // G, axis=1), sel, -INF)
    order = np.lexsort((np.where(bad.numpy()[:, None], 0.0, -l.numpy()), -sel), axis=1)[:, :k]
    none = torch.from_numpy(np.take_along_axis(sel, order, 1) == -INF)
    order = torch.from_numpy(order)
    w = s.gather(1, order).masked_fill(none, 0.0)
    if cfg.norm_topk_prob:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * float(torch.tensor(cfg.routed_scaling_factor, dtype=torch.float32))
    w[bad] = math.nan
    return order.masked_fill(none, -1).to(torch.int32), w


def route_weights(cfg, logits, idx):
    """The weights as a differentiable function of fp64 logits, experts held."""
    has = (idx >= 0) & (idx < logits.shape[1])
    at = torch.where(has, idx, 0).long()
    if cfg.norm_topk_prob and cfg.score_fn == "softmax":
        # the row's sum of exponentials cancels: a softmax of the chosen alone
        l = logits.gather(1, at)
        top = torch.where(has, l, -INF).max(1, keepdim=True)[0].detach()
        p = torch.exp(l - torch.where(top == -INF, 0.0, top))
    else:
        p = scores(logits, cfg.score_fn).gather(1, at)
    p = torch.where(has, p, 0.0)
    if cfg.norm_topk_prob:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(has.any(1, keepdim=True), total, 1.0)
    return p * float(torch.tensor(cfg.routed_scaling_factor, dtype=torch.float32))


def combine_backward(dout, y, row_of, w, dy):
    T, k = w.shape
    dout, dy, dw = dout.double(), dy.double().clone(), torch.zeros(T, k, dtype=torch.float64)
    for p, row in enumerate(row_of.tolist()):
        if 0 <= row < T * k:
            t, j = divmod(p, k)
            dy[row] = w[t, j].double() * dout[t]
            dw[t, j] = (dout[t] * y[row].double()).sum()
    return dy, dw


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(x, w, bias, residual, name):
    z = x.double() @ w.double().t()
    if bias is not None:
        z = z + bias.double()
    y = act(z, name)
    return z, y if residual is None else y + residual.double()


def linear_backward(dy, x, w, pre, name):
    g = dy.double()
    if name != "none":
        z = pre.double().clone().requires_grad_(True)
        g = torch.autograd.grad(act(z, name), z, g)[0]
    return g, g @ w.double(), g.t() @ x.double(), g.sum(0)
