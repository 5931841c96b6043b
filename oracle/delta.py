"""Double-precision reference of the gated delta rule (test infrastructure
only): the definition, token after token, and its gradient written out by hand.

Next to every result stands what its rounding errors are proportional to.  With
g <= 0 and beta |k|^2 <= 2 a step takes no norm of the state up, so an error made
at one token reaches later ones at most as large as it was made: the norms of
what the tokens add, faded like the state, bound the sum of all of them.  The same
holds going back: a token takes the gradient R of the state to e^g (R - beta R k k^T),
no larger in norm, and its own rounding adds beta |k|^2 |R|.  A product is off by
either factor's error times the other's norm.
"""
import torch

F64 = torch.float64


def _setup(q, k, v, g, beta, state, lengths):
    N, L, H, P = v.shape
    r = H // q.shape[2]
    q, k = (x.to(F64).repeat_interleave(r, 2) for x in (q, k))
    v, g, beta = v.to(F64), g.to(F64), beta.to(F64)
    n = torch.full((N,), L) if lengths is None else lengths.clamp(0, L)
    live = torch.arange(L)[None] < n[:, None]                      # [N, L]
    S = torch.zeros(N, H, P, q.shape[3], dtype=F64) if state is None else state.to(F64).clone()
    return q, k, v, g, beta, live, S


def _norm(x, dims=1):
    return x.flatten(x.dim() - dims).square().sum(-1).sqrt()


def _states(q, k, v, g, beta, live, S):
    """[(S', error, S, m)] of every token: the faded state, v - S' k, the new state and its errors' scale [N, H]."""
    m, out = _norm(S, 2), []
    for t in range(v.shape[1]):
        on = live[:, t, None]
        faded = torch.where(on[..., None, None], S * g[:, t].exp()[..., None, None], S)
        e = torch.where(on[..., None], v[:, t] - (faded * k[:, t, :, None]).sum(-1), torch.zeros((), dtype=F64))
        b = torch.where(on, beta[:, t], torch.zeros((), dtype=F64))
        S = torch.where(on[..., None, None], faded + (b[..., None] * e)[..., None] * k[:, t, :, None], S)
        kn = _norm(k[:, t])
        m = torch.where(on, m * g[:, t].exp() + beta[:, t].abs() * (_norm(v[:, t]) + _norm(faded, 2) * kn) * kn, m)
        out.append((faded, e, S, m))
    return out


def delta(q, k, v, g, beta, scale, state=None, lengths=None):
    """y, the last state, and the scales of their errors, [N, L, H, 1] and [N, H, 1, 1]."""
    q, k, v, g, beta, live, S = _setup(q, k, v, g, beta, state, lengths)
    y, my, m = torch.zeros_like(v), torch.zeros(v.shape[:3] + (1,), dtype=F64), _norm(S, 2)
    for t, (_, _, S, m) in enumerate(_states(q, k, v, g, beta, live, S)):
        y[:, t] = scale * (S * q[:, t, :, None]).sum(-1) * live[:, t, None, None]
        my[:, t, :, 0] = abs(scale) * m * _norm(q[:, t])
    return y, S, my, m[..., None, None]


def delta_grad(dy, q, k, v, g, beta, scale, state=None, lengths=None, dstate_out=None):
    """dicts of dq, dk, dv, dg, dbeta, dstate and of the scales of their errors."""
    G = q.shape[2]
    q, k, v, g, beta, live, S0 = _setup(q, k, v, g, beta, state, lengths)
    N, L, H, P = v.shape
    steps = _states(q, k, v, g, beta, live, S0)
    R = torch.zeros_like(S0) if dstate_out is None else dstate_out.to(F64).clone()
    mr, m0 = _norm(R, 2), _norm(S0, 2)
    d = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v), "dg": torch.zeros_like(g),
         "dbeta": torch.zeros_like(g)}
    mag = {n: torch.zeros_like(g) for n in d}
    dy = torch.where(live[..., None, None], dy.to(F64), torch.zeros((), dtype=F64)) * scale
    for t in reversed(range(L)):
        faded, e, S, ms = steps[t]
        on = live[:, t, None].to(F64)
        kn, qn, vn, b = _norm(k[:, t]), _norm(q[:, t]), _norm(v[:, t]), beta[:, t].abs()
        d["dq"][:, t] = (S * dy[:, t, ..., None]).sum(-2)
        mag["dq"][:, t] = _norm(dy[:, t]) * ms
        R = R + dy[:, t, ..., None] * q[:, t, :, None]
        # R's own norm and that of its error (what was added so far), e's, the faded state's
        mr = mr + on * _norm(dy[:, t]) * qn
        rn, en, sn, me = _norm(R, 2), _norm(e), _norm(faded, 2), vn + kn * ms
        rk = (R * k[:, t, :, None]).sum(-1)
        d["dbeta"][:, t] = on * (rk * e).sum(-1)
        mag["dbeta"][:, t] = on * kn * (mr * en + rn * me)
        d["dv"][:, t] = on[..., None] * beta[:, t][..., None] * rk
        mag["dv"][:, t] = on * b * kn * mr
        u = beta[:, t][..., None] * e
        d["dk"][:, t] = on[..., None] * ((R * u[..., None]).sum(-2) - (faded * d["dv"][:, t, ..., None]).sum(-2))
        mag["dk"][:, t] = on * b * (mr * (en + kn * sn) + rn * (me + kn * ms))
        back = R - d["dv"][:, t, ..., None] * k[:, t, :, None]
        d["dg"][:, t] = on * (back * faded).sum((-1, -2))
        # besides, the terms that cross the token's decay are summed: what is added behind it times what was added in
        # front, which may cancel.  They take the roundings of their own products and decays, an eighth of a state's.
        mag["dg"][:, t] = on * (mr * sn + rn * ms + mr * ms / 8)
        live4 = live[:, t, None, None, None]
        R = torch.where(live4, back * g[:, t].exp()[..., None, None], R)
        mr = torch.where(live[:, t, None], (mr + b * kn * kn * rn) * g[:, t].exp(), mr)
    group = lambda x: x.unflatten(2, (G, H // G)).sum(3)
    d["dq"], d["dk"] = group(d["dq"]), group(d["dk"])
    mag["dq"], mag["dk"] = group(mag["dq"])[..., None], group(mag["dk"])[..., None]
    mag["dv"] = mag["dv"][..., None]
    d["dstate"], mag["dstate"] = R, mr[..., None, None]
    return d, mag


def step(q, k, v, g, beta, scale, state):
    """One token: y (N, H, P), the new state, and the scales of their errors."""
    y, S, my, m = delta(q[:, None], k[:, None], v[:, None], g[:, None], beta[:, None], scale, state)
    return y[:, 0], S, my[:, 0], m
