"""Double-precision reference of the group norm (test infrastructure only): the
definition and its gradient written out by hand, next to each result the scale of
its rounding errors (sums of the terms' absolute values)."""
import math

import torch

F64 = torch.float64


def _act(name, v):
    """The activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * c, c + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    return v, torch.ones_like(v)


def _parts(x, w, bias, lengths, center, per_token, eps):
    x, w = x.to(F64), w.to(F64)
    N, L, G, C = x.shape
    n = torch.full((N,), L) if lengths is None else lengths.clamp(0, L).long()
    live = (torch.arange(L)[None] < n[:, None])[..., None, None]
    x = torch.where(live, x, torch.zeros((), dtype=F64))
    dims = (3,) if per_token else (1, 3)
    count = torch.tensor(float(C), dtype=F64) if per_token else (n.clamp(min=1) * C).to(F64)[:, None, None, None]
    mean = x.sum(dims, keepdim=True) / count
    d = torch.where(live, x - mean, torch.zeros((), dtype=F64)) if center else x
    r = 1 / (d.square().sum(dims, keepdim=True) / count + eps).sqrt()
    xhat = d * r
    b = torch.zeros_like(w) if bias is None else bias.to(F64)
    # x and the mean are what a difference is rounded by
    rough = (x.abs() + (mean.abs() if center else 0)) * r
    return live, dims, count, r, xhat, w, b, rough


def norm(x, w, bias=None, gate=None, lengths=None, act="none", center=True, per_token=False, eps=1e-5):
    """y and the scale of its errors."""
    live, _, _, _, xhat, w, b, rough = _parts(x, w, bias, lengths, center, per_token, eps)
    v, mv = xhat * w + b, rough * w.abs() + b.abs()
    zero = torch.zeros((), dtype=F64)
    if gate is not None:
        z = torch.where(live, gate.to(F64), zero)
        y, mag = v * _act(act, z)[0], mv * (1 + z.abs())
    else:
        y, mag = _act(act, v)[0], mv
    return torch.where(live, y, zero), torch.where(live, mag, zero)


def norm_grad(dy, x, w, bias=None, gate=None, lengths=None, act="none", center=True, per_token=False, eps=1e-5):
    """dicts of dx, dw, dbias, dgate and of the scales of their errors."""
    live, dims, count, r, xhat, w, b, rough = _parts(x, w, bias, lengths, center, per_token, eps)
    zero = torch.zeros((), dtype=F64)
    dy = torch.where(live, dy.to(F64), zero)
    v, mv = xhat * w + b, rough * w.abs() + b.abs()
    if gate is not None:
        z = torch.where(live, gate.to(F64), zero)
        a, da = _act(act, z)
        d, dz, far = dy * a, dy * v * da, 1 + z.abs()
    else:
        d, dz, far = dy * _act(act, v)[1], torch.zeros_like(x, dtype=F64), 1 + mv
    md = dy.abs() * far
    g = {"dw": (d * xhat).sum((0, 1)), "dbias": d.sum((0, 1)), "dgate": dz}
    m = {"dw": (md * rough).sum((0, 1)), "dbias": md.sum((0, 1)), "dgate": dy.abs() * mv * far}
    d, md = d * w, md * w.abs()
    m1, m2 = d.sum(dims, keepdim=True) / count, (d * xhat).sum(dims, keepdim=True) / count
    g["dx"] = torch.where(live, r * (d - (m1 if center else 0) - xhat * m2), zero)
    m["dx"] = torch.where(live, r * (md + md.sum(dims, keepdim=True) / count + rough * (md * rough).sum(dims, keepdim=True) / count), zero)
    return g, m
