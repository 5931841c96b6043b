"""Double-precision reference of the sequence operators (test infrastructure
only): the causal convolution and the selective scan from their definitions,
token after token, and their gradients written out by hand.

magnitude=True evaluates every sum with the absolute values of its terms: what
the rounding errors of a computed result are proportional to.
"""
import torch

F64 = torch.float64


def _lens(lengths, N, L):
    if lengths is None:
        return [L] * N
    return [min(max(int(v), 0), L) for v in lengths]


def causal(x, w, bias, silu, state=None, lengths=None):
    """(y, state_out, v): v the sum before the activation."""
    x, w = x.to(F64), w.to(F64)
    N, L, C = x.shape
    F = w.shape[1]
    old = torch.zeros(N, F - 1, C, dtype=F64) if state is None else state.to(F64)
    y, v, out = torch.zeros(N, L, C, dtype=F64), torch.zeros(N, L, C, dtype=F64), old.clone()
    for n, m in enumerate(_lens(lengths, N, L)):
        h = torch.cat([old[n], x[n, :m]])
        acc = torch.zeros(m, C, dtype=F64) if bias is None else bias.to(F64).expand(m, C).clone()
        for k in range(F):
            acc = acc + w[:, k] * h[k:k + m]
        v[n, :m] = acc
        y[n, :m] = acc * torch.sigmoid(acc) if silu else acc
        out[n] = h[m:]
    return y, out, v


def causal_grad(dy, x, w, bias, silu, state=None, lengths=None, dstate_out=None, magnitude=False):
    """dict of dx, dw, dbias, dstate."""
    N, L, C = x.shape
    F = w.shape[1]
    _, _, v = causal(x, w, bias, silu, state, lengths)
    s = torch.sigmoid(v)
    d = dy.to(F64) * (s + v * s * (1 - s)) if silu else dy.to(F64).clone()
    x, w = x.to(F64), w.to(F64)
    old = torch.zeros(N, F - 1, C, dtype=F64) if state is None else state.to(F64)
    last = torch.zeros(N, F - 1, C, dtype=F64) if dstate_out is None else dstate_out.to(F64)
    if magnitude:
        d, x, w, old, last = d.abs(), x.abs(), w.abs(), old.abs(), last.abs()
    g = {"dx": torch.zeros(N, L, C, dtype=F64), "dw": torch.zeros(C, F, dtype=F64), "dbias": torch.zeros(C, dtype=F64),
         "dstate": torch.zeros(N, F - 1, C, dtype=F64)}
    for n, m in enumerate(_lens(lengths, N, L)):
        h = torch.cat([old[n], x[n, :m]])
        dh = torch.zeros_like(h)
        dh[m:] += last[n]
        for k in range(F):
            dh[k:k + m] += w[:, k] * d[n, :m]
            g["dw"][:, k] += (d[n, :m] * h[k:k + m]).sum(0)
        g["dbias"] += d[n, :m].sum(0)
        g["dx"][n, :m] = dh[F - 1:]
        g["dstate"][n] = dh[:F - 1]
    return g


def _scan_inputs(x, dt, A, B, C, dt_bias, softplus, lengths):
    N, L, H, P = x.shape
    G = B.shape[2]
    raw = dt.to(F64) + (0 if dt_bias is None else dt_bias.to(F64))
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw
    live = torch.zeros(N, L, dtype=F64)
    for n, m in enumerate(_lens(lengths, N, L)):
        live[n, :m] = 1
    heads = lambda v: v.to(F64).repeat_interleave(H // G, 2)
    zero = torch.zeros((), dtype=F64)
    inside = lambda v: torch.where(live.reshape(N, L, *[1] * (v.dim() - 2)) > 0, v, zero)
    return inside(x.to(F64)), inside(step), raw, A.to(F64), inside(heads(B)), inside(heads(C)), live


def scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=True, state=None, lengths=None, magnitude=False):
    """(y, state_out)."""
    N, L, H, P = x.shape
    S = B.shape[3]
    x, step, _, A, B, C, live = _scan_inputs(x, dt, A, B, C, dt_bias, softplus, lengths)
    D = torch.zeros(H, dtype=F64) if D is None else D.to(F64)
    h = torch.zeros(N, H, P, S, dtype=F64) if state is None else state.to(F64).clone()
    if magnitude:
        x, B, C, D, h = x.abs(), B.abs(), C.abs(), D.abs(), h.abs()
    y = torch.zeros(N, L, H, P, dtype=F64)
    for t in range(L):
        h = torch.exp(A * step[:, t])[..., None, None] * h + \
            (step[:, t, :, None] * x[:, t])[..., None] * B[:, t, :, None, :]
        y[:, t] = (h * C[:, t, :, None, :]).sum(-1) + D[:, None] * x[:, t]
    return y * live[..., None, None], h


def scan_grad(dy, x, dt, A, B, C, D=None, dt_bias=None, softplus=True, state=None, lengths=None, dstate_out=None,
              magnitude=False):
    """dict of dx, ddt, dA, dB, dC, dD, ddt_bias, dstate, and of dl (the gradient of A step), e (of step, by way of the
    input) and step, the step sizes."""
    N, L, H, P = x.shape
    G, S = B.shape[2], B.shape[3]
    x, step, raw, A, B, C, live = _scan_inputs(x, dt, A, B, C, dt_bias, softplus, lengths)
    D = torch.zeros(H, dtype=F64) if D is None else D.to(F64)
    dy = torch.where(live[..., None, None] > 0, dy.to(F64), torch.zeros((), dtype=F64))
    h = torch.zeros(N, H, P, S, dtype=F64) if state is None else state.to(F64).clone()
    u = torch.zeros(N, H, P, S, dtype=F64) if dstate_out is None else dstate_out.to(F64).clone()
    if magnitude:
        x, B, C, D, dy, h, u = x.abs(), B.abs(), C.abs(), D.abs(), dy.abs(), h.abs(), u.abs()
    hs = [h]
    a = torch.exp(A * step)
    for t in range(L):
        h = a[:, t, :, None, None] * h + (step[:, t, :, None] * x[:, t])[..., None] * B[:, t, :, None, :]
        hs.append(h)
    dx, dl, e = torch.zeros_like(x), torch.zeros_like(step), torch.zeros_like(step)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    for t in reversed(range(L)):
        dC[:, t] = (dy[:, t][..., None] * hs[t + 1]).sum(2)
        u = u + dy[:, t][..., None] * C[:, t, :, None, :]
        into = (u * B[:, t, :, None, :]).sum(-1)                    # of dt x
        dx[:, t] = step[:, t, :, None] * into + D[:, None] * dy[:, t]
        e[:, t] = (into * x[:, t]).sum(-1)
        dB[:, t] = ((step[:, t, :, None] * x[:, t])[..., None] * u).sum(2)
        dl[:, t] = a[:, t] * (hs[t] * u).sum((-1, -2))
        u = a[:, t, :, None, None] * u
    mult = A.abs() if magnitude else A
    ddt = (dl * mult + e) * (torch.sigmoid(raw) if softplus else 1.0) * live[..., None]
    groups = lambda v: v.unflatten(2, (G, H // G)).sum(3)
    return {"dx": dx * live[..., None, None], "ddt": ddt, "dA": (dl * step).sum((0, 1)), "dB": groups(dB),
            "dC": groups(dC), "dD": (dy * x).sum((0, 1, 3)), "ddt_bias": ddt.sum((0, 1)), "dstate": u,
            "dl": dl, "e": e, "step": step}
